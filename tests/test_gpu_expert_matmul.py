"""ep_quantize_rows and ep_expert_matmul against the plain 64-bit forms.

Tolerances.  Codes: |q - v / scale| <= 1/2 plus the error of v * inv, which for
|v * inv| <= 127 and at most 10 float32 roundings (SwiGLU: exp, sum, division,
product; the reciprocal and its product) is below 127 * 10 * 2^-24 * 1.5 <
2e-4; scales: the same roundings, relative.
Products: sums of |x||w| below 2^24 are exact integers in any order; above,
each of the Kd / 16 additions of 16-term partial sums rounds (or cuts) to 24
bits: (Kd / 16 + 4) 2^-23 of the sum of magnitudes.  The two scales add three
float32 roundings, the output's type one more."""
import numpy as np
import pytest
import torch

import _expert_ref as ref
import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
CONTIG, MASKED = ep.EP_LAYOUT_CONTIG, ep.EP_LAYOUT_MASKED
CODE_TOL = 0.5 + 2e-4
SCALE_RTOL = 10 * 2.0 ** -24 * 1.5


def rows_of(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.rand((rows, 1), generator=g) * 5
    if rows > 2:
        x[1] = 0.0
        x[2] *= 1e-30
    return x.to(dtype)


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 48), (3, 1024), (7, 1040), (3, 2064), (5, 2880),
                                       (2, 7168), (3, 8192), (2, 8208), (2, 20000)])
def test_quantize_against_plain(rows, cols, dtype, act):
    wide = 2 * cols if act == ep.EP_ACT_SWIGLU else cols
    x = rows_of(rows, wide, dtype, rows + cols)
    q, s = ep.ep_quantize_rows(x.cuda(), act=act)
    v = x.double().numpy()
    if act == ep.EP_ACT_SWIGLU:
        v = ref.swiglu(v)
        v[np.abs(v) < 2.0 ** -149] = 0.0  # float32 holds nothing smaller
    want, scale = ref.quantize(v)
    q, s = q.double().cpu().numpy(), s.double().cpu().numpy()
    ok = np.abs(v).max(1) > 1e-30  # below, products of float32 lose bits to the denormal range
    np.testing.assert_allclose(s[ok], scale[ok], rtol=SCALE_RTOL)
    assert np.abs(q[ok] - want[ok]).max() <= CODE_TOL
    assert np.abs(q).max() <= 127
    zero = np.abs(v).max(1) == 0
    assert (q[zero] == 0).all() and (s[zero] == 1).all()


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU])
@pytest.mark.parametrize("rows,cols", [(4096, 512), (4099, 528), (4097, 1056), (4098, 1440), (4096, 1536), (4096, 1552), (4096, 2064), (4100, 2880),
                                       (2, 272), (2, 1440), (2, 2576), (2, 4112), (2, 5136), (2, 9216), (2, 16384)])
def test_quantize_block_shapes(rows, cols, act):
    """Lengths that leave threads or vectors of a block idle, by a warp and by a block a row."""
    x = rows_of(rows, 2 * cols if act == ep.EP_ACT_SWIGLU else cols, torch.bfloat16, cols)
    q, s = ep.ep_quantize_rows(x.cuda(), act=act)
    v = x.double().numpy()
    if act == ep.EP_ACT_SWIGLU:
        v = ref.swiglu(v)
    want, scale = ref.quantize(v)
    ok = np.abs(v).max(1) > 1e-30
    np.testing.assert_allclose(s.double().cpu().numpy()[ok], scale[ok], rtol=SCALE_RTOL)
    assert np.abs(q.double().cpu().numpy()[ok] - want[ok]).max() <= CODE_TOL


def test_quantize_rounds_ties_to_even():
    x = torch.zeros((1, 32))
    x[0, 0] = 127.0
    x[0, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5])
    q, s = ep.ep_quantize_rows(x.cuda())
    assert float(s[0]) == 1.0
    assert q[0, :9].tolist() == [127, 0, 2, 2, 0, -2, -2, 126, -126]


@pytest.mark.parametrize("cols", [64, 512, 2048, 20000])
def test_quantize_tiny_rows(cols):
    """Rows near the bottom of float32's range: 127 over their largest value
    would overflow.  Scales below the normal range hold fewer bits, so codes are
    compared with v / (max|v| / 127) and the scale within a denormal unit."""
    g = torch.Generator().manual_seed(cols)
    x = torch.randn((5, cols), generator=g) * torch.tensor([[1e-30], [1e-34], [1e-37], [1e-40], [1e-44]])
    x[:, 3] = 0.0
    q, s = ep.ep_quantize_rows(x.cuda())
    v = x.double().numpy()
    want, scale = ref.quantize(v)
    assert np.abs(q.double().cpu().numpy() - want).max() <= CODE_TOL
    assert (np.abs(s.double().cpu().numpy() - scale) <= SCALE_RTOL * scale + 2.0 ** -149).all()


@pytest.mark.parametrize("layout", [CONTIG, MASKED])
def test_quantize_skips_rows_without_a_token(layout):
    E, cap, cols = 4, 6, 64
    offs = torch.tensor([0, 3, 3, 11, 13], dtype=torch.int32)
    rows = E * cap
    x = rows_of(rows, cols, torch.bfloat16, 3)
    q = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -5.0, device="cuda")
    ep.ep_quantize_rows(x.cuda(), expert_offsets=offs.cuda(), layout=layout, cap=cap, q=q, scales=s)
    all_q, all_s = ep.ep_quantize_rows(x.cuda())
    for r in range(rows):
        if layout == CONTIG:
            valid = r < 13
        else:
            valid = r % cap < int(offs[r // cap + 1] - offs[r // cap])
        if valid:
            assert torch.equal(q[r], all_q[r]) and s[r] == all_s[r]
        else:
            assert (q[r] == 99).all() and s[r] == -5.0


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def ints(shape, seed, full):
    g = np.random.default_rng(seed)
    if full:
        return g.integers(-128, 128, shape).astype(np.int8)
    return np.clip(np.rint(g.normal(0, 30, shape)), -127, 127).astype(np.int8)


def run_case(counts, Nc, Kd, layout, cap, gather, out_dtype, seed=0, full=True):
    E = len(counts)
    offs = offsets(counts)
    n = int(offs[-1])
    g = np.random.default_rng(seed + 1)
    rows = E * cap if layout == MASKED else n + 3  # contiguous: a few rows past the last expert's
    xr = max(1, n // 2) if gather else rows
    x, w = ints((xr, Kd), seed + 2, full), ints((E, Nc, Kd), seed + 3, full)
    xs = g.uniform(0.01, 0.05, xr).astype(np.float32)
    ws = g.uniform(0.001, 0.01, (E, Nc)).astype(np.float32)
    src = None
    if gather:
        src = g.integers(0, xr, rows if layout == CONTIG else max(n, 1)).astype(np.int32)
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    out = torch.full((rows, Nc), 123.0, dtype=out_dtype, device="cuda")
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    ep.ep_expert_matmul(c(x), c(xs), c(w), c(ws), c(offs), layout=layout, cap=cap, row_src=c(src),
                        out=out, status=status)
    want, mag, written = ref.matmul(x, xs, w, ws, offs, layout, cap, src, rows)
    got = out.double().cpu().numpy()
    assert int(status) == 0
    assert (got[~written] == 123.0).all()
    tol = 4 * 2.0 ** -24 * np.abs(want) + 1e-30
    small = Kd * 128 * 128 < 2 ** 24
    if not small:
        tol = tol + (Kd / 16 + 4) * 2.0 ** -23 * mag
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    bad = np.abs(got - want)[written] > tol[written]
    assert not bad.any(), (bad.sum(), bad.size, np.abs(got - want)[written].max())
    return got


COUNTS = {
    "one row": [1],
    "one expert": [37],
    "empty first and last": [0, 5, 0, 17, 1, 0],
    "none": [0, 0, 0],
    "one holds all": [0, 0, 300, 0],
    "ragged": [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 5],
    "tiles": [255, 256, 257, 0, 512, 513],
}


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("Nc,Kd", [(1, 16), (33, 64), (128, 128), (257, 272), (300, 1040)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_matmul_contiguous(counts, Nc, Kd, out_dtype):
    run_case(COUNTS[counts], Nc, Kd, CONTIG, 0, False, out_dtype)


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("cap", [1, 16, 40, 300])
@pytest.mark.parametrize("gather", [False, True])
def test_matmul_masked(counts, cap, gather):
    run_case(COUNTS[counts], 130, 144, MASKED, cap, gather, torch.float32, seed=cap)


@pytest.mark.parametrize("counts", ["one row", "ragged", "tiles"])
@pytest.mark.parametrize("Nc,Kd", [(64, 512), (515, 2880)])
def test_matmul_gathered(counts, Nc, Kd):
    run_case(COUNTS[counts], Nc, Kd, CONTIG, 0, True, torch.bfloat16, seed=5, full=False)


@pytest.mark.parametrize("rows", [1, 2, 3, 8, 9, 16, 24, 48, 65, 96, 130, 200, 300])
def test_matmul_one_expert_any_rows(rows):
    run_case([rows], 384, 400, CONTIG, 0, False, torch.float32, seed=rows)


@pytest.mark.parametrize("counts,Nc,Kd", [
    ([40] * 40, 640, 144),            # more tiles than CTAs, narrow
    ([130, 100, 0, 159] * 8, 1100, 400),
    ([300, 257] * 10, 1100, 144),     # wide tiles
    ([700, 1, 0, 90] * 6, 1030, 272),
    ([5], 2000, 1440),                # few tiles: K divided among CTAs
    ([64], 256, 2064),
    ([50, 0, 3], 200, 528),
    ([17] * 6, 130, 384),
])
@pytest.mark.parametrize("layout,gather,out_dtype", [(CONTIG, True, torch.bfloat16), (CONTIG, False, torch.float32),
                                                     (MASKED, True, torch.float32)])
def test_matmul_many_and_few_tiles(counts, Nc, Kd, layout, gather, out_dtype):
    run_case(counts, Nc, Kd, layout, max(counts) if layout == MASKED else 0, gather, out_dtype, seed=Kd)


@pytest.mark.parametrize("Kd", [16, 32, 112, 128, 144, 2032, 7168, 65536])
@pytest.mark.parametrize("rows", [3, 150])
def test_matmul_lengths(Kd, rows):
    if Kd == 65536 and rows > 3:
        rows = 40
    run_case([rows, 0, 2], 140, Kd, CONTIG, 0, False, torch.float32, seed=Kd)


def test_matmul_sums_below_2_to_24_are_exact():
    """Kd = 1024 of the largest codes: the integer sum, bit for bit."""
    for rows in (2, 200):
        x = torch.full((rows, 1008), -128, dtype=torch.int8, device="cuda")
        w = torch.full((1, 200, 1008), -128, dtype=torch.int8, device="cuda")
        x[:, 5] = 1
        w[0, :, 9] = 127
        out = ep.ep_expert_matmul(x, torch.ones(rows, device="cuda"), w,
                                  torch.ones((1, 200), device="cuda"),
                                  torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                                  out_dtype=torch.float32)
        want = (x.double() @ w[0].double().T)
        assert torch.equal(out.double(), want)


@pytest.mark.parametrize("rows", [6, 400])
def test_matmul_source_rows_out_of_range_are_zero(rows):
    E, Nc, Kd = 2, 96, 128
    x = torch.from_numpy(ints((5, Kd), 1, True)).cuda()
    w = torch.from_numpy(ints((E, Nc, Kd), 2, True)).cuda()
    src = torch.arange(rows, dtype=torch.int32) % 5
    src[0], src[rows // 2], src[rows - 1] = -1, 5, 2 ** 31 - 1
    offs = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    out = ep.ep_expert_matmul(x, torch.ones(5, device="cuda"), w, torch.ones((E, Nc), device="cuda"),
                              offs, row_src=src.cuda(), out_dtype=torch.float32)
    good = (src >= 0) & (src < 5)
    assert (out.cpu()[~good] == 0).all()
    for r in torch.nonzero(good).flatten().tolist():
        e = 0 if r < rows // 2 else 1
        assert torch.equal(out[r].double(), w[e].double() @ x[int(src[r])].double())


@pytest.mark.parametrize("layout,cap", [(CONTIG, 0), (MASKED, 10)])
def test_matmul_malformed_offsets_stay_inside(layout, cap):
    """Offsets that are negative, decreasing or past the rows: nothing outside
    the output is written (the buffer's surroundings keep their values)."""
    E, Nc, Kd = 4, 64, 64
    rows = 40
    x = torch.from_numpy(ints((rows, Kd), 1, True)).cuda()
    w = torch.from_numpy(ints((E, Nc, Kd), 2, True)).cuda()
    for offs in ([0, 2 ** 31 - 1, 5, -7, 100], [-50, 10, 8, 39, 41], [0, 90, 90, 90, 90],
                 [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]):
        buf = torch.full((rows + 64, Nc), 55.0, device="cuda")
        out = buf[32:32 + rows]
        ep.ep_expert_matmul(x, torch.ones(rows, device="cuda"), w,
                            torch.ones((E, Nc), device="cuda"),
                            torch.tensor(offs, dtype=torch.int32, device="cuda"), layout=layout,
                            cap=cap, out=out)
        torch.cuda.synchronize()
        assert (buf[:32] == 55).all() and (buf[32 + rows:] == 55).all()


def test_matmul_runs_on_the_given_stream_in_a_graph_and_repeats():
    counts = [40, 0, 130, 7]
    offs = torch.from_numpy(offsets(counts)).cuda()
    n, Nc, Kd = sum(counts), 200, 320
    x = torch.from_numpy(ints((n, Kd), 1, False)).cuda()
    w = torch.from_numpy(ints((4, Nc, Kd), 2, False)).cuda()
    xs, ws = torch.rand(n, device="cuda"), torch.rand((4, Nc), device="cuda")
    out = torch.empty((n, Nc), dtype=torch.bfloat16, device="cuda")
    want = ep.ep_expert_matmul(x, xs, w, ws, offs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ep.ep_expert_matmul(x, xs, w, ws, offs, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.ep_expert_matmul(x, xs, w, ws, offs, out=out)
    x.copy_(torch.from_numpy(ints((n, Kd), 7, False)))
    for _ in range(3):
        out.zero_()
        g.replay()
        want = ep.ep_expert_matmul(x, xs, w, ws, offs)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_matmul_first_call_of_a_process_inside_a_capture(tmp_path):
    """Nothing that a first call looks up keeps it from being captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
import combine_ep_route_topk_gb300 as ep
x = torch.randint(-9, 9, (64, 128), device="cuda").to(torch.int8)
w = torch.randint(-9, 9, (2, 96, 128), device="cuda").to(torch.int8)
offs = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
one, ws = torch.ones(64, device="cuda"), torch.ones((2, 96), device="cuda")
outs = [torch.zeros((64, 96), device="cuda") for _ in range(2)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ep.ep_expert_matmul(x, one, w, ws, offs, out=outs[0])
g.replay()
torch.cuda.synchronize()
want = torch.cat([x[:40].double() @ w[0].double().T, x[40:].double() @ w[1].double().T])
assert torch.equal(outs[0].double(), want)
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("E,rows", [(1024, 2000), (16, 5000)])
def test_matmul_overlapping_offsets_stay_inside(E, rows):
    """Every expert claims every row: more tiles than rows, no write outside."""
    Nc, Kd = 8, 16
    x = torch.from_numpy(ints((rows, Kd), 1, True)).cuda()
    w = torch.from_numpy(ints((E, Nc, Kd), 2, True)).cuda()
    offs = torch.zeros(E + 1, dtype=torch.int32)
    offs[1::2] = 2 ** 31 - 1
    buf = torch.full((rows + 64, Nc), 55.0, device="cuda")
    ep.ep_expert_matmul(x, torch.ones(rows, device="cuda"), w, torch.ones((E, Nc), device="cuda"),
                        offs.cuda(), out=buf[32:32 + rows])
    torch.cuda.synchronize()
    assert (buf[:32] == 55).all() and (buf[32 + rows:] == 55).all()


@pytest.mark.slow
@pytest.mark.parametrize("rows", [3, 60])
def test_matmul_weights_past_4_gib(rows):
    """Weight and scale offsets beyond 32 bits: the last expert's rows."""
    E, Nc, Kd = 40, 8192, 16384
    w = torch.empty((E, Nc, Kd), dtype=torch.int8, device="cuda")
    w.random_(-128, 128, generator=torch.Generator("cuda").manual_seed(3))
    x = torch.from_numpy(ints((rows, Kd), 4, False)).cuda()
    offs = torch.zeros(E + 1, dtype=torch.int32)
    offs[E - 1], offs[E] = rows // 3, rows
    offs[2:E - 1] = rows // 3
    ws = torch.rand((E, Nc), device="cuda")
    out = ep.ep_expert_matmul(x, torch.ones(rows, device="cuda"), w, ws, offs.cuda(),
                              out_dtype=torch.float32)
    for r in range(rows):
        e = 1 if r < rows // 3 else E - 1
        want = (w[e].double() @ x[r].double()) * ws[e].double()
        mag = (w[e].double().abs() @ x[r].double().abs()) * ws[e].double()
        assert ((out[r].double() - want).abs() <= (Kd / 16 + 4) * 2.0 ** -23 * mag).all()


@pytest.mark.slow
def test_matmul_output_past_2_to_31_elements():
    E, Nc, Kd, rows = 2, 8192, 16, 270000
    x = torch.empty((rows, Kd), dtype=torch.int8, device="cuda").random_(-128, 128)
    w = torch.empty((E, Nc, Kd), dtype=torch.int8, device="cuda").random_(-128, 128)
    offs = torch.tensor([0, 1000, rows], dtype=torch.int32, device="cuda")
    out = ep.ep_expert_matmul(x, torch.ones(rows, device="cuda"), w, torch.ones((E, Nc), device="cuda"),
                              offs)
    for r in (0, 999, 1000, 262143, 262144, 262145, rows - 1):
        e = 0 if r < 1000 else 1
        assert torch.equal(out[r], (w[e].double() @ x[r].double()).float().to(torch.bfloat16))
