"""Grouped products (forward, gradients, 8-bit) and the 8-bit row quantiser
against plain sums in 64 bits.

Tolerances, from the arithmetic alone.  Products of 16-bit or e4m3 operands are
exact in fp32.  A sum of n of them in fp32, in any order and with every
partial sum rounded or truncated, is off by at most n * 2^-23 * S, where S is
the sum of the products' magnitudes (a truncation is off by less than one step,
2^-23 of the partial sum, and each partial sum is at most S).  Rounding to the
output's type adds eps / 2 of the value (half its smallest subnormal step for
results near zero).  The 8-bit product's two scale multiplications add 2^-23
each, inside the same count (n + 4)."""
import numpy as np
import pytest
import torch

import bit_quantized_moe_route_b200 as moe

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ws(cuda_device):
    return moe.alloc_grouped_workspace(cuda_device)


def gen(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def normal(g, dtype, *shape, std=1.0):
    return torch.empty(shape, dtype=dtype, device=g.device).normal_(0.0, std, generator=g)


def offsets_of(counts, dev, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + start, dtype=torch.int32, device=dev)


def strided(g, dtype, rows, cols, pad, shift=0):
    """[rows, cols] with `pad` more elements per row, `shift` elements into its buffer."""
    buf = normal(g, dtype, rows * (cols + pad) + shift)
    return buf[shift:].view(rows, cols + pad)[:, :cols]


def close(got, ref, mag, n, label=""):
    """got against the 64-bit ref; mag = sum of the products' magnitudes, n = how many there are."""
    eps = torch.finfo(got.dtype).eps / 2 if got.dtype != FP else 2.0 ** -24
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    tol = (n + 4) * 2.0 ** -23 * mag * (1 + eps) + eps * ref.abs() + tiny
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (label, int(bad.sum()), (err / tol).nan_to_num(1e9).max().item(),
                                 bad.nonzero()[:4].tolist())


def reference(op, a, b, off, experts):
    """(values, magnitudes) in 64 bits over the whole output; rows of no expert are NaN."""
    off = [0, a.shape[0]] if off is None else off.tolist()
    a, b = a.double(), b.double()
    if op == "dw":
        out = torch.zeros(experts, a.shape[1], b.shape[1], dtype=torch.float64, device=a.device)
        mag = torch.zeros_like(out)
        for e in range(experts):
            u, v = a[off[e]:off[e + 1]], b[off[e]:off[e + 1]]
            out[e], mag[e] = u.t() @ v, u.abs().t() @ v.abs()
        return out, mag
    cols = b.shape[1] if op == "mm" else b.shape[2]
    out = torch.full((a.shape[0], cols), float("nan"), dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(out)
    for e in range(experts):
        w = b[e].t() if op == "mm" else b[e]
        u = a[off[e]:off[e + 1]]
        out[off[e]:off[e + 1]], mag[off[e]:off[e + 1]] = u @ w, u.abs() @ w.abs()
    return out, mag


def run_op(op, counts, n_in, n_out, dtype, out, dev, ws, pad=0, start=0, ld_pad=0, shift=0, seed=0, dense=False):
    """One call on random inputs, checked whole: values, rows of no expert, and no device error."""
    g = gen(seed + 1000 * n_in + n_out, dev)
    experts, rows = len(counts), start + int(sum(counts)) + pad
    off = None if dense else offsets_of(counts, dev, start)
    w = normal(g, dtype, experts * n_out * n_in + shift, std=0.05)[shift:].view(experts, n_out, n_in)
    x, dy = strided(g, dtype, rows, n_in, ld_pad, shift), strided(g, dtype, rows, n_out, ld_pad, shift)
    if op == "dw":
        y = torch.full((experts, n_out, n_in), 7.0, dtype=out, device=dev)
        moe.grouped_mm_dw(dy, x, off, y, ws)
        n = torch.tensor(counts, device=dev, dtype=torch.float64)[:, None, None]
    else:
        cols = n_out if op == "mm" else n_in
        y = torch.full((rows, cols + ld_pad), 7.0, dtype=out, device=dev)[:, :cols]
        if op == "mm":
            moe.grouped_mm(x, w, off, y, ws)
        else:
            moe.grouped_mm_dx(dy, w, off, y, ws)
        n = n_in if op == "mm" else n_out
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == 0
    ref, mag = reference(op, dy if op != "mm" else x, x if op == "dw" else w, off, experts)
    label = (op, counts, n_in, n_out)
    if op == "dw":
        close(y, ref, mag, n, label)
    else:
        inside = torch.zeros(rows, dtype=torch.bool, device=dev)
        inside[start:rows - pad] = True
        close(y[inside], ref[inside], mag[inside], n, label)
        assert bool((y[~inside] == 7.0).all())
        assert ld_pad == 0 or bool((y.as_strided((rows, ld_pad), (cols + ld_pad, 1), cols) == 7.0).all())
    return y


OPS = ["mm", "dx", "dw"]
RAGGED = [0, 1, 5, 0, 17, 64, 65, 130, 0]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, HF), (BF, FP), (HF, FP)])
@pytest.mark.parametrize("n_in,n_out", [(256, 128), (64, 320), (72, 40), (8, 8), (136, 264)])
def test_ragged(cuda_device, ws, op, dtype, out, n_in, n_out):
    run_op(op, RAGGED, n_in, n_out, dtype, out, cuda_device, ws)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("n_in,n_out", [(1, 1), (33, 100), (257, 129), (100, 64), (64, 100), (7, 300)])
def test_odd_widths(cuda_device, ws, op, n_in, n_out):
    run_op(op, RAGGED, n_in, n_out, BF, BF, cuda_device, ws)
    run_op(op, [3], n_in, n_out, HF, FP, cuda_device, ws, dense=True)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("counts", [[1], [0], [0, 0, 0], [1, 0, 0, 1], [256], [257], [511, 0, 513], [16] * 40, [1] * 300,
                                    [2000]])
def test_row_counts(cuda_device, ws, op, counts):
    run_op(op, counts, 192, 256, BF, FP, cuda_device, ws)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("ld_pad,shift", [(8, 0), (24, 8), (3, 0), (0, 1), (5, 3)])
def test_strides_and_alignment(cuda_device, ws, op, ld_pad, shift):
    run_op(op, [5, 0, 70, 33], 128, 192, BF, BF, cuda_device, ws, ld_pad=ld_pad, shift=shift)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("pad,start", [(1, 0), (77, 0), (0, 5), (300, 130)])
def test_rows_of_no_expert_stay(cuda_device, ws, op, pad, start):
    run_op(op, [9, 0, 140, 1], 128, 256, HF, HF, cuda_device, ws, pad=pad, start=start)


@pytest.mark.parametrize("op", OPS)
def test_one_matrix_without_offsets(cuda_device, ws, op):
    for rows in (1, 2, 31, 300):
        run_op(op, [rows], 512, 384, BF, BF, cuda_device, ws, dense=True, seed=rows)


@pytest.mark.parametrize("op", OPS)
def test_long_sums_of_few_outputs(cuda_device, ws, op):
    """Few outputs and a long contracted dimension: the work is split along it."""
    counts = [1, 3] if op != "dw" else [9000, 1, 4100]
    wide = {"mm": (8192, 64), "dx": (64, 8192), "dw": (64, 72)}[op]
    run_op(op, counts, *wide, BF, FP, cuda_device, ws)
    run_op(op, counts, *wide, HF, HF, cuda_device, ws)


@pytest.mark.parametrize("op", OPS)
def test_many_experts(cuda_device, ws, op):
    counts = np.random.default_rng(4).integers(0, 4, 1024).tolist()
    run_op(op, counts, 64, 72, BF, BF, cuda_device, ws)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("op,counts,wide,other", [
    ("mm", [300, 0, 1, 77, 256, 513, 40, 33] * 5, 2348, 1024), ("mm", [90] * 40, 2304, 200), ("mm", [3] * 80, 1100, 64),
    ("dx", [300, 0, 1, 77, 256, 513, 40, 33] * 5, 2344, 1024), ("dx", [90] * 40, 2304, 200), ("dx", [3] * 80, 1096, 64),
    ("dw", [300, 0, 1, 77, 256, 513, 40, 1300] * 5, 1000, 520), ("dw", [65] * 40, 776, 328), ("dw", [0] * 100, 512, 512)])
def test_many_tiles(cuda_device, ws, dtype, op, counts, wide, other):
    """Enough tiles for the widest ones: their odd last halves, short and long sums, whole and split tiles."""
    n_in, n_out = {"mm": (other, wide), "dx": (wide, other), "dw": (other, wide)}[op]
    run_op(op, counts, n_in, n_out, dtype, dtype, cuda_device, ws, pad=5, start=3 if op != "dw" else 0)


@pytest.mark.parametrize("op", ["mm", "dx", "fp8"])
@pytest.mark.parametrize("seed", range(3))
def test_mixed_tile_widths(cuda_device, ws, op, seed):
    """Row counts that make tiles of every width follow one another many times over in one launch: narrow and wide
    accumulators share tensor memory in changing patterns."""
    g = np.random.default_rng(seed)
    counts = [int(g.choice([1, 20, 33, 64, 65, 128, 129, 200, 256, 300])) for _ in range(60)]
    if op == "fp8":
        run_fp8(counts, 256, 2048, BF, cuda_device, ws)
    else:
        run_op(op, counts, *((128, 2048) if op == "mm" else (2048, 128)), BF, BF if seed else FP, cuda_device, ws)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("aligned", [True, False])
def test_same_bits_every_time(cuda_device, ws, op, aligned):
    n_in = 2048 if aligned else 2047
    a = run_op(op, [3, 40, 0, 7], n_in, 320, BF, FP, cuda_device, ws)
    for _ in range(3):
        assert torch.equal(a, run_op(op, [3, 40, 0, 7], n_in, 320, BF, FP, cuda_device, ws))


@pytest.mark.parametrize("n_in", [128, 100])
def test_nothing_leaks_between_experts(cuda_device, ws, n_in):
    """NaN and infinity in rows of no expert, in another expert's rows and in weights without rows stay there."""
    g = gen(3, cuda_device)
    counts, n_out = [5, 0, 20, 9], 136
    off = offsets_of(counts, cuda_device)
    x, dy = normal(g, BF, 50, n_in), normal(g, BF, 50, n_out)
    w = normal(g, BF, 4, n_out, n_in)
    clean_x, clean_dy, clean_w = x.clone(), dy.clone(), w.clone()
    for t in (x, dy):
        t[34:] = float("nan")
        t[5:25] = float("inf")
    w[1] = float("nan")
    w[2, 0, 0] = float("inf")
    keep = [r for r in range(34) if not 5 <= r < 25]
    for op, a, ca, cols in (("mm", x, clean_x, n_out), ("dx", dy, clean_dy, n_in)):
        y = torch.zeros(50, cols, dtype=FP, device=cuda_device)
        (moe.grouped_mm if op == "mm" else moe.grouped_mm_dx)(a, w, off, y, ws)
        ref, mag = reference(op, ca, clean_w, off, 4)
        close(y[keep], ref[keep], mag[keep], n_in if op == "mm" else n_out, op)
        assert bool((~torch.isfinite(y[5:25])).all()) and bool((y[34:] == 0).all())
    dw = torch.empty(4, n_out, n_in, dtype=FP, device=cuda_device)
    moe.grouped_mm_dw(dy, x, off, dw, ws)
    ref, mag = reference("dw", clean_dy, clean_x, off, 4)
    for e in (0, 1, 3):
        close(dw[e], ref[e], mag[e], 50, ("dw", e))
    assert not bool(torch.isfinite(dw[2]).any())
    assert moe.read_device_error(ws) == 0


@pytest.mark.parametrize("n_in", [128, 127])
def test_bad_offsets(cuda_device, ws, n_in):
    x, w = torch.ones(20, n_in, dtype=BF, device=cuda_device), torch.ones(3, 64, n_in, dtype=BF, device=cuda_device)
    dy = torch.ones(20, 64, dtype=BF, device=cuda_device)
    for bad in ([-1, 3, 5, 9], [0, 5, 4, 9], [0, 5, 9, 21], [0, 2 ** 31 - 1, 3, 4], [5, 2, 9, 20], [0, 0, 0, -2 ** 31]):
        off = torch.tensor(bad, dtype=torch.int32, device=cuda_device)
        y = torch.full((20, 64), 7.0, dtype=BF, device=cuda_device)
        dx = torch.full((20, n_in), 7.0, dtype=BF, device=cuda_device)
        dw = torch.full((3, 64, n_in), 7.0, dtype=BF, device=cuda_device)
        for call, out in ((lambda: moe.grouped_mm(x, w, off, y, ws), y), (lambda: moe.grouped_mm_dx(dy, w, off, dx, ws), dx),
                          (lambda: moe.grouped_mm_dw(dy, x, off, dw, ws), dw)):
            call()
            assert moe.read_device_error(ws) == 6, bad
            assert bool((out == 7.0).all())
    off = torch.tensor([0, 5, 5, 20], dtype=torch.int32, device=cuda_device)
    y = torch.empty(20, 64, dtype=BF, device=cuda_device)
    moe.grouped_mm(x, w, off, y, ws)
    assert moe.read_device_error(ws) == 0 and bool((y == n_in).all())   # 127 and 128 are bf16 values


def test_overlap_and_host_memory_refused(cuda_device, ws):
    w = torch.zeros(1, 64, 64, dtype=BF, device=cuda_device)
    x = torch.zeros(8, 64, dtype=BF, device=cuda_device)
    with pytest.raises(moe.MoEError, match="overlaps x"):
        moe.grouped_mm(x, w, None, x, ws)
    with pytest.raises(moe.MoEError, match="overlaps w"):
        moe.grouped_mm(x, w, None, w[0, :8], ws)
    with pytest.raises(ValueError):
        moe.grouped_mm(x.cpu(), w, None, x, ws)
    with pytest.raises(moe.MoEError) as e:
        moe.grouped_mm(x, w, None, torch.zeros_like(x), ws[:4096])
    assert e.value.status == 3
    s = torch.zeros(1, 8, device=cuda_device)
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.quant_fp8(x, x.view(-1).view(torch.uint8)[:512].view(8, 64), s)


def test_column_ranges_of_one_buffer(cuda_device, ws):
    """Input and output side by side in one buffer are apart; ranges that share a column are not."""
    g = gen(12, cuda_device)
    buf = normal(g, BF, 40, 320)
    w = normal(g, BF, 1, 128, 192, std=0.1)
    x, y = buf[:, :192], buf[:, 192:]
    ref, mag = reference("mm", x, w, None, 1)
    keep = x.clone()
    moe.grouped_mm(x, w, None, y, ws)
    close(y, ref, mag, 192)
    assert torch.equal(x, keep)
    dx = buf[:, 128:]
    moe.grouped_mm_dx(buf[:, :128], w, None, dx, ws)             # the other order
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.grouped_mm(buf[:, :192], w, None, buf[:, 191:319], ws)
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.grouped_mm(buf[:, 100:292], w, None, buf[:, :128], ws)


def test_range_of_fp16(cuda_device, ws):
    """Sums beyond fp16 become infinite; subnormal operands count."""
    for n_in in (64, 63):
        x, w = torch.full((4, n_in), 300.0, dtype=HF, device=cuda_device), torch.zeros(1, 16, n_in, dtype=HF, device=cuda_device)
        w[0, 0], w[0, 1] = 300.0, -300.0
        w[0, 2, 0] = 2.0 ** -24                                    # the smallest fp16 subnormal
        y = torch.zeros(4, 16, dtype=HF, device=cuda_device)
        moe.grouped_mm(x, w, None, y, ws)
        assert bool((y[:, 0] == float("inf")).all()) and bool((y[:, 1] == float("-inf")).all())
        assert bool((y[:, 2] == torch.tensor(300 * 2.0 ** -24, dtype=HF, device=cuda_device)).all())
        assert bool((y[:, 3:] == 0).all())


FIRST_CALL = """
import torch, bit_quantized_moe_route_b200 as moe
dev = torch.device("cuda:0")
ws = moe.alloc_grouped_workspace(dev)
off = torch.tensor([0, 3, 3, 10], dtype=torch.int32, device=dev)
side = torch.cuda.Stream(dev)
for n_in in (128, 127):
    x = torch.ones(10, n_in, dtype=torch.bfloat16, device=dev)
    w = torch.ones(3, 64, n_in, dtype=torch.bfloat16, device=dev)
    y, dx = torch.zeros(10, 64, device=dev), torch.zeros(10, n_in, device=dev)
    dw = torch.full((3, 64, n_in), 5.0, device=dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):      # the process's first calls
        moe.grouped_mm(x, w, off, y, ws)
        moe.grouped_mm_dx(x.new_ones(10, 64), w, off, dx, ws)
        moe.grouped_mm_dw(x.new_ones(10, 64), x, off, dw, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert bool((y == n_in).all()) and bool((dx == 64).all())
    assert dw[0].unique().tolist() == [3.0] and dw[1].unique().tolist() == [0.0] and dw[2].unique().tolist() == [7.0]
assert moe.read_device_error(ws) == 0
print("ok")
"""


def test_first_call_in_a_capture(cuda_device):
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_streams_and_graphs(cuda_device):
    """Two streams with a workspace each, and a captured call replayed on new inputs."""
    g = gen(8, cuda_device)
    counts = [2, 0, 30, 1]
    off = offsets_of(counts, cuda_device)
    w = normal(g, BF, 4, 256, 1024, std=0.05)
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    spaces = [moe.alloc_grouped_workspace(cuda_device) for _ in range(2)]
    xs = [normal(g, BF, 33, 1024) for _ in range(2)]
    ys = [torch.zeros(33, 256, dtype=FP, device=cuda_device) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, sp, x, y in zip(streams, spaces, xs, ys):
            moe.grouped_mm(x, w, off, y, sp, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        ref, mag = reference("mm", x, w, off, 4)
        close(y, ref, mag, 1024)
    graph = torch.cuda.CUDAGraph()
    x, y = xs[0].clone(), torch.zeros_like(ys[0])
    dy, dx, dw = normal(g, BF, 33, 256), torch.zeros(33, 1024, dtype=BF, device=cuda_device), torch.zeros_like(w)
    with torch.cuda.graph(graph):
        moe.grouped_mm(x, w, off, y, spaces[0])
        moe.grouped_mm_dx(dy, w, off, dx, spaces[0])
        moe.grouped_mm_dw(dy, x, off, dw, spaces[0])
    for seed in range(3):
        x.copy_(normal(gen(100 + seed, cuda_device), BF, 33, 1024))
        graph.replay()
        ref, mag = reference("mm", x, w, off, 4)
        close(y, ref, mag, 1024)
        ref, mag = reference("dx", dy, w, off, 4)
        close(dx, ref, mag, 256)
        ref, mag = reference("dw", dy, x, off, 4)
        close(dw, ref, mag, 33)
    new = torch.tensor([0, 10, 10, 11, 33], dtype=torch.int32, device=cuda_device)   # other row ranges, same graph
    off.copy_(new)
    graph.replay()
    ref, mag = reference("mm", x, w, new, 4)
    close(y, ref, mag, 1024)
    assert [moe.read_device_error(s) for s in spaces] == [0, 0]


def test_gradients_by_differences(cuda_device, ws):
    """The loss is linear in x and in W, so a difference quotient along any direction is exact but for rounding."""
    g = gen(21, cuda_device)
    counts, n_in, n_out = [3, 0, 18, 7], 96, 80
    off = offsets_of(counts, cuda_device)
    x, w = normal(g, HF, 28, n_in), normal(g, HF, 4, n_out, n_in, std=0.1)
    dy = normal(g, HF, 28, n_out)

    def loss(x_, w_):
        y = torch.empty(28, n_out, dtype=FP, device=cuda_device)
        moe.grouped_mm(x_, w_, off, y, ws)
        return (y.double() * dy.double()).sum()

    dx, dw = torch.empty(28, n_in, dtype=FP, device=cuda_device), torch.empty(4, n_out, n_in, dtype=FP, device=cuda_device)
    moe.grouped_mm_dx(dy, w, off, dx, ws)
    moe.grouped_mm_dw(dy, x, off, dw, ws)
    # directions of +-1/4 on values rounded to multiples of 2^-6: sums with them are exact in fp16
    x, w = (x * 64).round() / 64, (w * 64).round() / 64
    moe.grouped_mm_dx(dy, w, off, dx, ws)
    moe.grouped_mm_dw(dy, x, off, dw, ws)
    size = reference("mm", x.abs() + 0.25, w.abs() + 0.25, off, 4)[1]
    tol = 2 * (n_in + n_out + 40) * 2.0 ** -23 * float((size * dy.double().abs()).sum())
    for _ in range(3):
        v = torch.randint(0, 2, x.shape, generator=g, device=cuda_device).to(HF) * 0.5 - 0.25
        assert abs(float(loss(x + v, w) - loss(x, w) - (dx.double() * v.double()).sum())) <= tol
        v = torch.randint(0, 2, w.shape, generator=g, device=cuda_device).to(HF) * 0.5 - 0.25
        assert abs(float(loss(x, w + v) - loss(x, w) - (dw.double() * v.double()).sum())) <= tol


# ------------------------------------------------------------------ 8 bits
def quant_reference(x):
    """Codes and scales by the formula, each step rounded once to fp32."""
    rows, n = x.shape
    groups = (n + 127) // 128
    v = torch.zeros(rows, groups * 128, dtype=FP, device=x.device)
    v[:, :n] = x.float()
    v = v.view(rows, groups, 128)
    a = v.abs().amax(2).clamp(min=448 * 2.0 ** -126)
    top = torch.full_like(a, 448.0)
    codes = (v * (top / a)[:, :, None]).to(torch.float8_e4m3fn).view(rows, -1)[:, :n].contiguous()
    return codes, (a / top).t().contiguous()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,n,ld_pad,shift", [(1, 4096, 0, 0), (1, 1, 0, 0), (37, 1024, 0, 0), (5, 128, 8, 0),
                                                 (33, 144, 0, 0), (64, 100, 0, 0), (70, 513, 3, 1), (3, 2048, 0, 1),
                                                 (300, 16, 16, 8), (2, 1000, 0, 0)])
def test_quant(cuda_device, dtype, rows, n, ld_pad, shift):
    g = gen(rows + n, cuda_device)
    x = strided(g, dtype, rows, n, ld_pad, shift)
    x[0, : n // 2] = 0
    codes = torch.zeros(rows, n, dtype=torch.float8_e4m3fn, device=cuda_device)
    scales = torch.zeros((n + 127) // 128, rows, device=cuda_device)
    moe.quant_fp8(x, codes, scales)
    ref, s = quant_reference(x)
    assert torch.equal(scales, s)
    assert torch.equal(codes.view(torch.uint8), ref.view(torch.uint8))
    # half a step of the code, relative to the value: 2^-4, or 2^-10 of the scale among e4m3's subnormals;
    # the two fp32 roundings of the factor and product move a value by 2^-23 at most
    full = s.t().repeat_interleave(128, 1)[:, :n].double()
    err = (codes.double() * full - x.double()).abs()
    assert bool((err <= (2.0 ** -4 * (1 + 2.0 ** -10)) * x.double().abs() + 2.0 ** -10 * full * (1 + 2.0 ** -10)).all())


def test_quant_extremes(cuda_device):
    """Zeros, the smallest and largest values, and groups with an infinity or a NaN."""
    x = torch.zeros(8, 256, dtype=BF, device=cuda_device)
    x[1, 3] = 2.0 ** -133                       # a bf16 subnormal
    x[2, 130] = torch.finfo(BF).max
    x[2, 131] = -torch.finfo(BF).max
    x[3] = torch.linspace(-3, 3, 256).to(BF)
    x[4, 5], x[5, 200], x[6, 128] = float("inf"), float("nan"), float("-inf")
    x[4, 6] = 1.0
    for strip in (False, True):                 # 16-byte aligned rows, and odd ones
        v = x[:, 1:] if strip else x
        codes = torch.zeros(v.shape, dtype=torch.float8_e4m3fn, device=cuda_device)
        scales = torch.zeros(2, 8, device=cuda_device)
        moe.quant_fp8(v, codes, scales)
        ref, s = quant_reference(v)
        assert torch.equal(torch.isnan(scales), torch.isnan(s)) and torch.equal(scales.nan_to_num(1.0), s.nan_to_num(1.0))
        assert torch.equal(codes.float().nan_to_num(99.0), ref.float().nan_to_num(99.0))
        value = codes.float() * scales.t().repeat_interleave(128, 1)[:, :v.shape[1]]
        assert bool(torch.isnan(value[4, :128]).all()) and bool((value[4, 128:] == 0).all())
        assert bool(torch.isnan(value[5, 128:]).all()) and bool((value[5, :128] == 0).all())
        assert bool((value[0] == 0).all()) and bool(torch.isfinite(value[1:4]).all())


def fp8_inputs(g, experts, rows, n_in, n_out, ld_pad=0, shift=0):
    dev = g.device
    codes = torch.empty(rows * (n_in + ld_pad) + shift, dtype=torch.uint8, device=dev)
    codes = codes[shift:].view(rows, n_in + ld_pad)[:, :n_in]
    v = normal(g, FP, rows, n_in, std=100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes.copy_(v.view(torch.uint8))
    w = torch.empty(experts * n_out * n_in + shift, dtype=torch.uint8, device=dev)[shift:].view(experts, n_out, n_in)
    w.copy_(normal(g, FP, experts, n_out, n_in, std=100.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    gi, go = (n_in + 127) // 128, (n_out + 127) // 128
    sx = torch.exp(normal(g, FP, gi, rows, std=2.0)) * 0.01
    sw = torch.exp(normal(g, FP, experts, go, gi, std=2.0)) * 0.001
    return codes, sx, w, sw


def fp8_wide(codes, s, n_out=None):
    """Values of 8-bit rows ([groups, rows] scales) or weights (block scales) in 64 bits."""
    v = codes.view(torch.float8_e4m3fn).double() if codes.is_contiguous() else \
        codes.contiguous().view(torch.float8_e4m3fn).double()
    if v.dim() == 2:
        return v * s.t().repeat_interleave(128, 1)[:, :v.shape[1]].double()
    return v * s.repeat_interleave(128, 1)[:, :v.shape[1]].repeat_interleave(128, 2)[:, :, :v.shape[2]].double()


def run_fp8(counts, n_in, n_out, out, dev, ws, pad=0, ld_pad=0, shift=0, dense=False):
    g = gen(n_in + n_out, dev)
    experts, rows = len(counts), int(sum(counts)) + pad
    off = None if dense else offsets_of(counts, dev)
    codes, sx, w, sw = fp8_inputs(g, experts, rows, n_in, n_out, ld_pad, shift)
    y = torch.full((rows, n_out + ld_pad), 7.0, dtype=out, device=dev)[:, :n_out]
    moe.grouped_mm_fp8(codes, sx, w, sw, off, y, ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == 0
    ref, mag = reference("mm", fp8_wide(codes, sx), fp8_wide(w, sw), off, experts)
    used = rows - pad
    close(y[:used], ref[:used], mag[:used], n_in, ("fp8", counts, n_in, n_out))
    assert bool((y[used:] == 7.0).all())
    return y


@pytest.mark.parametrize("out", [BF, FP])
@pytest.mark.parametrize("n_in,n_out", [(256, 128), (128, 320), (144, 40), (16, 8), (640, 264), (1, 1), (100, 129),
                                        (300, 257)])
def test_fp8_ragged(cuda_device, ws, out, n_in, n_out):
    run_fp8(RAGGED, n_in, n_out, out, cuda_device, ws)


@pytest.mark.parametrize("counts", [[1], [0, 0], [256], [300, 0, 513], [1] * 300, [16] * 40])
def test_fp8_row_counts(cuda_device, ws, counts):
    run_fp8(counts, 384, 256, FP, cuda_device, ws, pad=3)


@pytest.mark.parametrize("out", [BF, FP])
@pytest.mark.parametrize("n_in,n_out", [(256, 128), (128, 320), (144, 40), (640, 264), (1024, 1000), (384, 33)])
def test_fp8_many_rows(cuda_device, ws, out, n_in, n_out):
    """Many rows per expert on average, uneven, with short and empty experts among them."""
    run_fp8([700, 0, 1, 513, 256, 255, 37, 900], n_in, n_out, out, cuda_device, ws, pad=9)
    run_fp8([1500], n_in, n_out, out, cuda_device, ws, dense=True)


@pytest.mark.parametrize("ld_pad,shift", [(16, 0), (48, 16), (3, 0), (0, 1), (16, 5)])
def test_fp8_strides_and_alignment(cuda_device, ws, ld_pad, shift):
    run_fp8([5, 0, 70, 33], 256, 192, torch.float16 if shift == 5 else BF, cuda_device, ws, ld_pad=ld_pad, shift=shift)


@pytest.mark.parametrize("rows", [1, 2, 33, 300])
def test_fp8_one_matrix(cuda_device, ws, rows):
    a = run_fp8([rows], 4096, 320, FP, cuda_device, ws, dense=True)
    assert torch.equal(a, run_fp8([rows], 4096, 320, FP, cuda_device, ws, dense=True))


def test_fp8_nan_stays_in_its_row(cuda_device, ws):
    g = gen(5, cuda_device)
    counts = [4, 30]
    off = offsets_of(counts, cuda_device)
    codes, sx, w, sw = fp8_inputs(g, 2, 40, 256, 136)
    ref, mag = reference("mm", fp8_wide(codes, sx), fp8_wide(w, sw), off, 2)
    codes[7, 3] = 0x7F
    sx[1, 9] = float("nan")
    codes[34:] = 0x7F
    sx[:, 34:] = float("nan")
    y = torch.zeros(40, 136, dtype=FP, device=cuda_device)
    moe.grouped_mm_fp8(codes, sx, w, sw, off, y, ws)
    keep = [r for r in range(34) if r not in (7, 9)]
    close(y[keep], ref[keep], mag[keep], 256)
    assert bool(torch.isnan(y[[7, 9]]).all()) and bool((y[34:] == 0).all())


# ----------------------------------------------------------- used together
def _routed(dev, T, d, E, k, seed):
    g = gen(seed, dev)
    dims = moe.make_dims(T, d, 128, E, k)
    wsl = moe.alloc_workspace(dims, dev)
    x = normal(g, BF, T, d)
    rw, rb = normal(g, FP, E, d, std=0.05), normal(g, FP, E, std=0.1)
    ids, wt = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    srt, inv = torch.empty(T * k, dtype=torch.int32, device=dev), torch.empty(T * k, dtype=torch.int32, device=dev)
    moe.route(dims, x, rw, rb, None, None, ids, wt, wsl)
    moe.permute(dims, ids, off, srt, inv, wsl)
    assert moe.read_device_error(wsl) == 0
    return g, dims, wsl, x, ids, wt, off, srt, inv


@pytest.mark.parametrize("T", [1, 45])
def test_layer_over_source_weights(cuda_device, ws, T):
    """route, permute, three 16-bit products with SwiGLU between them, combine: the layer before its weights are
    packed, against the same sums in 64 bits (intermediate rounding to bf16 included, so 2^-8 of each stage)."""
    d, f, E, k = 256, 128, 8, 3
    g, dims, wsl, x, ids, wt, off, srt, inv = _routed(cuda_device, T, d, E, k, 31)
    w1, w3 = normal(g, BF, E, f, d, std=0.05), normal(g, BF, E, f, d, std=0.05)
    w2 = normal(g, BF, E, d, f, std=0.05)
    xs = x[(srt // k).long()]
    h1, h3 = (torch.empty(T * k, f, dtype=FP, device=cuda_device) for _ in range(2))
    y = torch.empty(T * k, d, dtype=FP, device=cuda_device)
    moe.grouped_mm(xs, w1, off, h1, ws)
    moe.grouped_mm(xs, w3, off, h3, ws)
    h = (torch.nn.functional.silu(h1) * h3).to(BF)
    moe.grouped_mm(h, w2, off, y, ws)
    out = torch.empty(T, d, dtype=BF, device=cuda_device)
    moe.combine(dims, y, inv, wt, None, out)
    assert moe.read_device_error(ws) == 0
    ref, mag = torch.zeros(T, d, dtype=torch.float64, device=cuda_device), 0
    mag = torch.zeros_like(ref)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            a, b = w1[e].double() @ x[t].double(), w3[e].double() @ x[t].double()
            hh = torch.nn.functional.silu(a) * b
            ref[t] += float(wt[t, j]) * (w2[e].double() @ hh)
            mag[t] += float(wt[t, j]) * (w2[e].double().abs() @ hh.abs())
    # h is rounded to bf16 (2^-8 of each term, plus fp32 sums of 256 terms well below it), the output once more
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * 1.05 * mag + 2.0 ** -8 * ref.abs() + 1e-6).all())


def test_layer_over_8bit_weights(cuda_device, ws):
    """The gate projection of routed rows, quantised to 8 bits, over 8-bit weights."""
    T, d, E, k, f = 45, 256, 8, 3, 192
    g, dims, wsl, x, ids, wt, off, srt, inv = _routed(cuda_device, T, d, E, k, 32)
    _, _, w, sw = fp8_inputs(g, E, 1, d, f)
    xs = x[(srt // k).long()]
    codes = torch.empty(T * k, d, dtype=torch.float8_e4m3fn, device=cuda_device)
    sx = torch.empty(d // 128, T * k, device=cuda_device)
    moe.quant_fp8(xs, codes, sx)
    y = torch.empty(T * k, f, dtype=BF, device=cuda_device)
    moe.grouped_mm_fp8(codes, sx, w, sw, off, y, ws)
    assert moe.read_device_error(ws) == 0
    wide_w = fp8_wide(w, sw)
    ref, mag = reference("mm", fp8_wide(codes, sx), wide_w, off, E)
    close(y, ref, mag, d)
    # against the rows before quantisation: half a code step (2^-4 of the value, 2^-10 of the scale) of each term
    full, m = reference("mm", xs, wide_w, off, E)
    step = reference("mm", sx.t().repeat_interleave(128, 1), wide_w, off, E)[1]
    assert bool(((y.double() - full).abs() <= 2.0 ** -4 * 1.01 * m + 2.0 ** -10 * 1.01 * step +
                 (d + 4) * 2.0 ** -23 * 2 * m + 2.0 ** -8 * 1.1 * full.abs() + 2.0 ** -12 * m).all())


def test_training_step(cuda_device, ws):
    """Forward, both gradients and a step against torch's own gradient of the same loss in 64 bits."""
    g = gen(41, cuda_device)
    counts, n_in, n_out = [12, 0, 33, 3], 128, 96
    off = offsets_of(counts, cuda_device)
    x, w, t = normal(g, BF, 48, n_in), normal(g, BF, 4, n_out, n_in, std=0.05), normal(g, FP, 48, n_out)
    y = torch.empty(48, n_out, dtype=FP, device=cuda_device)
    moe.grouped_mm(x, w, off, y, ws)
    dy = (y - t).to(BF)
    dx, dw = torch.empty_like(x), torch.empty(4, n_out, n_in, dtype=FP, device=cuda_device)
    moe.grouped_mm_dx(dy, w, off, dx, ws)
    moe.grouped_mm_dw(dy, x, off, dw, ws)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    o = off.tolist()
    y64 = torch.cat([x64[o[e]:o[e + 1]] @ w64[e].t() for e in range(4)])
    (y64 * dy.double()).sum().backward()
    _, mag = reference("dx", dy, w, off, 4)
    close(dx, x64.grad, mag, n_out)
    _, mag = reference("dw", dy, x, off, 4)
    close(dw, w64.grad, mag, 48)
    assert moe.read_device_error(ws) == 0


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("n_in,n_out", [(65, 129), (79, 1343), (1031, 77), (72, 2047)])
def test_any_alignment_items(cuda_device, ws, op, n_in, n_out):
    """Tiles of one step and experts without rows in a row, tiles of many, in operands that start anywhere."""
    counts = [1, 0, 0, 0, 0, 0, 0, 2, 0, 0, 0, 300, 0, 1, 0, 0, 0, 0, 0, 37]
    for shift, ld_pad in ((0, 0), (1, 0), (7, 3)):
        run_op(op, counts, n_in, n_out, BF, FP if shift else BF, cuda_device, ws, ld_pad=ld_pad, shift=shift, pad=5)


@pytest.mark.parametrize("n_in,n_out", [(127, 65), (1000, 300), (129, 2047)])
def test_fp8_any_alignment_items(cuda_device, ws, n_in, n_out):
    for shift, ld_pad in ((0, 0), (1, 0), (9, 5)):
        run_fp8([1, 0, 0, 0, 0, 0, 2, 0, 200, 0, 1, 70], n_in, n_out, BF, cuda_device, ws, ld_pad=ld_pad, shift=shift, pad=2)


@pytest.mark.parametrize("n_in,pitch", [(128, 32776), (129, 32771)])
def test_rows_beyond_4_gib(cuda_device, ws, n_in, pitch):
    """Rows whose byte offsets pass 32 bits, in and out."""
    rows, n_out, dev = 70000, 40, cuda_device
    g = gen(3, dev)
    x = torch.empty(rows * pitch, dtype=BF, device=dev).view(rows, pitch)[:, 5 if n_in == 129 else 8:][:, :n_in]
    x.copy_(normal(g, BF, rows, n_in))
    y = torch.empty(rows * pitch, dtype=BF, device=dev).view(rows, pitch)[:, :n_out]
    off = offsets_of([rows - 300, 0, 300], dev)
    w, dy = normal(g, BF, 3, n_out, n_in, std=0.05), normal(g, BF, rows, n_out)
    moe.grouped_mm(x, w, off, y, ws)
    dw = torch.empty(3, n_out, n_in, dtype=FP, device=dev)
    moe.grouped_mm_dw(dy, x, off, dw, ws)
    dx = y.as_strided((rows, n_in), (pitch, 1), 64)
    moe.grouped_mm_dx(dy, w, off, dx, ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == 0
    ref, mag = reference("mm", x, w, off, 3)
    close(y, ref, mag, n_in)
    ref, mag = reference("dx", dy, w, off, 3)
    close(dx, ref, mag, n_out)
    ref, mag = reference("dw", dy, x, off, 3)
    close(dw, ref, mag, torch.tensor([rows - 300, 0, 300], device=dev)[:, None, None])


@pytest.mark.parametrize("n_in", [8192, 8191])
def test_weights_beyond_4_gib(cuda_device, ws, n_in):
    """Matrices whose byte offsets pass 32 bits: read by the products, written by their gradient."""
    E, n_out, dev = 40, 8192, cuda_device
    g = gen(4, dev)
    counts = [2] + [0] * (E - 2) + [3]
    off = offsets_of(counts, dev)
    w = torch.empty(E, n_out, n_in, dtype=BF, device=dev)
    w[0], w[E - 1] = normal(g, BF, n_out, n_in, std=0.05), normal(g, BF, n_out, n_in, std=0.05)
    x, dy = normal(g, BF, 5, n_in), normal(g, BF, 5, n_out)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    moe.grouped_mm(x, w, off, y, ws)
    moe.grouped_mm_dx(dy, w, off, dx, ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == 0
    for lo, hi, e in ((0, 2, 0), (2, 5, E - 1)):
        m = w[e].double()
        close(y[lo:hi], x[lo:hi].double() @ m.t(), x[lo:hi].double().abs() @ m.t().abs(), n_in)
        close(dx[lo:hi], dy[lo:hi].double() @ m, dy[lo:hi].double().abs() @ m.abs(), n_out)
    moe.grouped_mm_dw(dy, x, off, w, ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == 0
    assert not bool(w[1:E - 1].any())
    for lo, hi, e in ((0, 2, 0), (2, 5, E - 1)):
        u, v = dy[lo:hi].double(), x[lo:hi].double()
        close(w[e], u.t() @ v, u.abs().t() @ v.abs(), hi - lo)


@pytest.mark.parametrize("n_in", [136, 137])
def test_replays_on_another_stream(cuda_device, n_in):
    """A captured forward and both gradients, replayed beside an eager call with a workspace of its own."""
    dev, g = cuda_device, gen(9, cuda_device)
    counts, n_out = [3, 0, 130, 1, 40], 200
    off, rows = offsets_of(counts, dev), sum(counts)
    x, dy, w = normal(g, BF, rows, n_in), normal(g, BF, rows, n_out), normal(g, BF, 5, n_out, n_in, std=0.05)

    def run(ws, y, dx, dw):
        moe.grouped_mm(x, w, off, y, ws)
        moe.grouped_mm_dx(dy, w, off, dx, ws)
        moe.grouped_mm_dw(dy, x, off, dw, ws)

    def outs():
        return torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w)

    ws1, ws2 = moe.alloc_grouped_workspace(dev), moe.alloc_grouped_workspace(dev)
    want, got, other = outs(), outs(), outs()
    run(ws2, *want)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(ws1, *got)
    for _ in range(4):
        for t in got + other:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            run(ws2, *other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, other))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("shift", [0, 1])
def test_long_fp32_sums_do_not_drift(cuda_device, ws, op, shift):
    """fp32 outputs of long sums of positive products, operands aligned and not: no drift from an accumulator that
    truncates.

    Values are 1 + j/16, so products have 8 fractional bits and are below 4: a sum of 512 of them is below 2^11 and
    has 19 bits, exact however it is taken.  What is left are ordinary additions of such sums, one for each 512
    products and at most two more for each of up to 74 parts of a tile; each rounds a partial sum, at most the whole,
    to nearest: 2^-24 of it.  Taken in one truncating accumulator the same sums are several times as far off."""
    length, m, n = 65536, 2560, 2048
    g = gen(17 + shift, cuda_device)

    def values(*shape):
        count = int(np.prod(shape))
        v = torch.randint(0, 16, (count + shift,), generator=g, device=cuda_device).to(BF) / 16 + 1
        return v[shift:].view(shape)

    if op == "mm":
        x, w, y = values(m, length), values(1, n, length), torch.empty(m, n, dtype=FP, device=cuda_device)
        moe.grouped_mm(x, w, None, y, ws)
        ref = x.double() @ w[0].double().t()
    elif op == "dx":
        dy, w, y = values(m, length), values(1, length, n), torch.empty(m, n, dtype=FP, device=cuda_device)
        moe.grouped_mm_dx(dy, w, None, y, ws)
        ref = dy.double() @ w[0].double()
    else:
        dy, x, y = values(length, m), values(length, n), torch.empty(1, m, n, dtype=FP, device=cuda_device)
        moe.grouped_mm_dw(dy, x, None, y, ws)
        ref = (dy.double().t() @ x.double())[None]
    torch.cuda.synchronize()
    assert moe.read_device_error(ws) == 0
    err = ((y.double() - ref).abs() / ref).max().item()
    assert err <= (length / 512 + 2 * 74) * 2.0 ** -24, err


@pytest.mark.parametrize("counts,n_in", [([40, 3], 384), ([300, 500], 384), ([40, 3], 383)])
@pytest.mark.parametrize("a,b", [(-63, -63), (-126, 0), (100, -120), (127, -60), (60, 36), (-3, 99)])
def test_fp8_scales_of_any_size(cuda_device, ws, counts, n_in, a, b):
    """Scales near both ends of fp32 whose product is normal, one sign or the other, zeros and zero blocks among them."""
    g, rows, n_out, dev = gen(a + 2 * b + 500, cuda_device), sum(counts), 136, cuda_device
    codes, sx, w, sw = fp8_inputs(g, 2, rows, n_in, n_out)
    sx = torch.full_like(sx, 2.0 ** a) * (1 - 2.0 * (torch.arange(rows, device=dev) % 2))
    sw = torch.full_like(sw, 2.0 ** b)
    sx[1, ::3], sw[1, 0, 2] = 0.0, 0.0
    codes[5:9, :128] = 0
    sx[0, 5:9] = min(2.0 ** (127 - max(b, 0)), 2.0 ** 127)        # the largest for this b: the blocks are zero
    y = torch.zeros(rows, n_out, dtype=FP, device=dev)
    moe.grouped_mm_fp8(codes, sx, w, sw, offsets_of(counts, dev), y, ws)
    assert moe.read_device_error(ws) == 0 and bool(torch.isfinite(y).all())
    ref, mag = reference("mm", fp8_wide(codes, sx), fp8_wide(w, sw), offsets_of(counts, dev), 2)
    close(y, ref, mag, n_in)


@pytest.mark.parametrize("counts,n_in", [([40, 3], 384), ([300, 500], 384), ([40, 3], 383)])
def test_fp8_scales_with_a_subnormal_product(cuda_device, ws, counts, n_in):
    """The product is rounded to a multiple of 2^-149, off by 2^-150 at most; times a group's sum, at most
    128 * 448 * 448 < 2^24.7, that is 2^-125.3 a group.  The quantiser's scale of a block of zeros gives exact zeros."""
    g, rows, n_out, dev = gen(77, cuda_device), sum(counts), 136, cuda_device
    codes, sx, w, sw = fp8_inputs(g, 2, rows, n_in, n_out)
    sx, sw = torch.full_like(sx, 1.7 * 2.0 ** -70), torch.full_like(sw, 1.9 * 2.0 ** -71)
    codes[:, :128], sx[0], sw[:, :, 0] = 0, 2.0 ** -126, 0.3       # blocks of zeros
    y = torch.zeros(rows, n_out, dtype=FP, device=dev)
    off = offsets_of(counts, dev)
    moe.grouped_mm_fp8(codes, sx, w, sw, off, y, ws)
    ref, mag = reference("mm", fp8_wide(codes, sx), fp8_wide(w, sw), off, 2)
    assert bool(((y.double() - ref).abs() <= 2 * 2.0 ** -125.3 + (n_in + 4) * 2.0 ** -23 * mag).all())
    codes.zero_()
    moe.grouped_mm_fp8(codes, sx, w, sw, off, y, ws)
    assert bool((y == 0).all()) and moe.read_device_error(ws) == 0


def test_operands_in_the_workspace_are_refused(cuda_device):
    """The workspace is written while the operands are read: none of them may lie in it; behind its bytes they may."""
    size = moe.grouped_workspace_size()
    buf = torch.zeros(size + (1 << 16), dtype=torch.uint8, device=cuda_device)
    part = buf[size - 8192:size].view(BF)
    x, y, w = part[:512].view(8, 64), torch.zeros(8, 64, dtype=BF, device=cuda_device), part[:4096].view(1, 64, 64)
    free, sx, sw = torch.ones(1, 64, 64, dtype=BF, device=cuda_device), torch.ones(1, 8, device=cuda_device), \
        torch.ones(1, 1, 1, device=cuda_device)
    off = buf[size - 8:size].view(torch.int32)
    codes, wide = torch.zeros(8, 64, dtype=torch.uint8, device=cuda_device), buf[size - 4096:size].view(1, 64, 64)
    calls = {
        "x": [lambda: moe.grouped_mm(x, free, None, y, buf), lambda: moe.grouped_mm_dw(y, x, None, free, buf)],
        "w": [lambda: moe.grouped_mm(y.clone(), w, None, y, buf), lambda: moe.grouped_mm_dx(y.clone(), w, None, y, buf),
              lambda: moe.grouped_mm_fp8(codes, sx, wide, sw, None, y, buf)],
        "dy": [lambda: moe.grouped_mm_dx(x, free, None, y, buf), lambda: moe.grouped_mm_dw(x, y, None, free, buf)],
        "expert_offsets": [lambda: moe.grouped_mm(y.clone(), free, off, y, buf)],
        "x_scales": [lambda: moe.grouped_mm_fp8(codes, part[:16].view(FP).view(1, 8), wide.clone(), sw, None, y, buf)],
        "w_scales": [lambda: moe.grouped_mm_fp8(codes, sx, wide.clone(), part[:2].view(FP).view(1, 1, 1), None, y, buf)]}
    for name, group in calls.items():
        for call in group:
            with pytest.raises(moe.MoEError, match=rf"ws overlaps {name}\)"):
                call()
    after = buf[size:size + 1024].view(BF).view(8, 64)
    after.fill_(1)
    moe.grouped_mm(after, free, None, y, buf)
    assert bool((y == 64).all()) and moe.read_device_error(buf) == 0


def whole(g, dtype, most, *shape):
    return torch.randint(-most, most + 1, shape, generator=g, device=g.device).to(dtype)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("length", [8192, 8191, 65536, 65535])
def test_long_sums_exactly(cuda_device, ws, op, dtype, length):
    """Whole numbers up to 4: every partial sum is one below 2^20 and exact in fp32, however it is taken, so that a
    product lost or counted twice anywhere in a long sum shows."""
    g, wide, rows = gen(length, cuda_device), 264, 77
    off = offsets_of([30, 0, 47], cuda_device)
    if op == "dw":
        off = offsets_of([length - 4100, 0, 4100], cuda_device)
        dy, x = whole(g, dtype, 4, length, wide), whole(g, dtype, 4, length, 135)
        y = torch.empty(3, wide, 135, dtype=FP, device=cuda_device)
        moe.grouped_mm_dw(dy, x, off, y, ws)
        ref, _ = reference("dw", dy, x, off, 3)
    elif op == "mm":
        x, w = whole(g, dtype, 4, rows, length), whole(g, dtype, 4, 3, wide, length)
        y = torch.empty(rows, wide, dtype=FP, device=cuda_device)
        moe.grouped_mm(x, w, off, y, ws)
        ref, _ = reference("mm", x, w, off, 3)
    else:
        dy, w = whole(g, dtype, 4, rows, length), whole(g, dtype, 4, 3, length, wide - length % 2)
        y = torch.empty(rows, wide - length % 2, dtype=FP, device=cuda_device)
        moe.grouped_mm_dx(dy, w, off, y, ws)
        ref, _ = reference("dx", dy, w, off, 3)
    assert moe.read_device_error(ws) == 0
    assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("n_in,pitch", [(128, 32776), (129, 32771)])
def test_rows_beyond_4_gib_exactly(cuda_device, ws, n_in, pitch):
    """Rows whose byte offsets pass 32 bits, of -1, 0 and 1: sums are exact in fp32 and, of 128 products, in bf16."""
    rows, n_out, dev = 70000, 40, cuda_device
    g, counts = gen(6, dev), [60000, 0, 10000]
    x = torch.empty(rows * pitch, dtype=BF, device=dev).view(rows, pitch)[:, 5 if n_in == 129 else 8:][:, :n_in]
    x.copy_(whole(g, BF, 1, rows, n_in))
    y = torch.empty(rows * pitch, dtype=BF, device=dev).view(rows, pitch)[:, :n_out]
    off, w, dy = offsets_of(counts, dev), whole(g, BF, 1, 3, n_out, n_in), whole(g, BF, 1, rows, n_out)
    dw, dx = torch.empty(3, n_out, n_in, dtype=FP, device=dev), y.as_strided((rows, n_in), (pitch, 1), 64)
    moe.grouped_mm(x, w, off, y, ws)
    moe.grouped_mm_dx(dy, w, off, dx, ws)
    moe.grouped_mm_dw(dy, x, off, dw, ws)
    assert moe.read_device_error(ws) == 0
    for op, got, a, b in (("mm", y, x, w), ("dx", dx, dy, w), ("dw", dw, dy, x)):
        assert torch.equal(got.double(), reference(op, a, b, off, 3)[0]), op


@pytest.mark.parametrize("counts,n_in,n_out", [([70], 65536, 136), ([70], 65535, 136), ([900], 65536, 264),
                                               ([20, 0, 50, 3], 8192, 129)])
def test_fp8_long_sums_exactly(cuda_device, ws, counts, n_in, n_out):
    """Whole numbers up to 4 and scales of 1/2, 1 and 2: sums up to 2^22 in steps of a quarter, exact in fp32."""
    g, rows, E, dev = gen(n_in + n_out, cuda_device), sum(counts), len(counts), cuda_device
    gi, go = (n_in + 127) // 128, (n_out + 127) // 128

    def codes(*shape):
        return whole(g, FP, 4, *shape).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales(*shape):
        return 2.0 ** whole(g, FP, 1, *shape)                     # 1/2, 1, 2

    x, w, sx, sw = codes(rows, n_in), codes(E, n_out, n_in), scales(gi, rows), scales(E, go, gi)
    y = torch.empty(rows, n_out, dtype=FP, device=dev)
    off = offsets_of(counts, dev)
    moe.grouped_mm_fp8(x, sx, w, sw, off, y, ws)
    assert moe.read_device_error(ws) == 0
    assert torch.equal(y.double(), reference("mm", fp8_wide(x, sx), fp8_wide(w, sw), off, E)[0])
