"""ep_expert_matmul_fp8 against the plain 64-bit form.

With codes that are small integers and scales that are powers of two every product
and sum is exact in float32, so that float32 outputs are compared bit for bit: that
shows every index, tile and block.  With codes over the whole range the bound is
_fp8_ref.matmul_tol's, on the sum of the products' magnitudes."""
import numpy as np
import pytest
import torch

import _fp8_ref as ref
import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
CONTIG, MASKED = ep.EP_LAYOUT_CONTIG, ep.EP_LAYOUT_MASKED
BF, F32 = torch.bfloat16, torch.float32


def small_codes(shape, g):
    """Codes of integers -8 .. 8."""
    v = torch.randint(-8, 9, shape, generator=g).float()
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def wide_codes(shape, g):
    """Codes of normal values scaled so that the largest are near 448."""
    v = (torch.randn(shape, generator=g) * 120).clamp(-448, 448)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def powers(shape, g):
    return 2.0 ** torch.randint(-1, 2, shape, generator=g).float()


def problem(counts, Nc, Kd, seed, exact, x_rows=None, cap=0, layout=CONTIG):
    g = torch.Generator().manual_seed(seed)
    E = len(counts)
    offs = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    rows = E * cap if layout == MASKED else int(offs[-1])
    n = rows if x_rows is None else x_rows
    codes = small_codes if exact else wide_codes
    kb, nb = ref.nblocks(Kd), ref.nblocks(Nc)
    if exact:
        xs, ws = powers((n, kb), g), powers((E, nb, kb), g)
    else:
        xs, ws = (0.5 + torch.rand((n, kb), generator=g)) / 120, (0.5 + torch.rand((E, nb, kb), generator=g)) / 120
    src = None
    if x_rows is not None:
        src = torch.randint(0, max(1, n), (int(offs[-1]),), generator=g, dtype=torch.int32)
    return dict(x=codes((n, Kd), g), xs=xs, w=codes((E, Nc, Kd), g), ws=ws, offs=offs, layout=layout,
                cap=cap, src=src, rows=rows)


def run(p, out_dtype=F32, out=None, status=None):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    if out is None:
        out = torch.full((p["rows"], p["w"].shape[1]), -77.0, dtype=out_dtype, device="cuda")
    return ep.ep_expert_matmul_fp8(c(p["x"]), c(p["xs"]), c(p["w"]), c(p["ws"]), c(p["offs"]),
                                   layout=p["layout"], cap=p["cap"], row_src=c(p["src"]), out=out,
                                   status=status)


def want_of(p):
    src = None if p["src"] is None else p["src"].numpy()
    return ref.matmul(p["x"].numpy(), p["xs"].numpy(), p["w"].numpy(), p["ws"].numpy(),
                      p["offs"].numpy(), p["layout"], p["cap"], src, p["rows"])


def check_exact(p):
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    got = run(p, status=status).double().cpu().numpy()
    want, mag, written = want_of(p)
    assert int(status) == 0
    assert mag.max(initial=0.0) < 2.0 ** 22  # multiples of 1/4 below 2^22: exact in any order
    np.testing.assert_array_equal(got[written], want[written])
    assert (got[~written] == -77.0).all()


def check_near(p, out_dtype):
    got = run(p, out_dtype).double().cpu().numpy()
    want, mag, written = want_of(p)
    rel_mag, rel = ref.matmul_tol(p["w"].shape[2], out_dtype == BF)
    assert (np.abs(got - want) <= rel_mag * mag + rel * np.abs(want))[written].all()
    assert (got[~written] == float(torch.tensor(-77.0, dtype=out_dtype))).all()


COUNTS = [
    ([1], 64, 128), ([1], 1, 16), ([0, 0, 3, 0], 130, 272), ([8] * 8, 256, 1024),
    ([1] * 12, 300, 400), ([127, 128, 129], 128, 144), ([40, 0, 300, 7], 520, 640),
    ([255, 256, 257, 1], 264, 256), ([1000], 384, 528), ([17] * 40, 72, 112),
    ([5, 600, 0, 0, 2, 64, 65], 1000, 1008), ([3] * 200, 8, 32), ([513, 31], 257, 2064),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,Nc,Kd", COUNTS)
def test_exact_sums_contiguous(counts, Nc, Kd, gather):
    check_exact(problem(counts, Nc, Kd, Nc + Kd, True, x_rows=37 if gather else None))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,Nc,Kd,cap", [
    ([1], 64, 128, 1), ([0, 5, 9, 2], 136, 272, 4), ([8] * 8, 256, 1024, 8), ([30, 0, 3], 520, 400, 200),
    ([300, 10, 290], 264, 656, 256), ([64] * 6, 500, 1008, 64), ([2] * 33, 130, 144, 130),
])
def test_exact_sums_masked(counts, Nc, Kd, cap, gather):
    check_exact(problem(counts, Nc, Kd, Nc + cap, True, x_rows=53 if gather else None, cap=cap,
                        layout=MASKED))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,Nc,Kd,cap", [
    ([300, 1, 0, 129] * 12, 1000, 272, 0),  # tiles for every SM, of an expert's rows in even parts
    ([257] * 30, 1544, 112, 0),             # one block of K a tile
    ([128, 200, 40, 260] * 20, 520, 656, 256),
    ([100] * 40, 1023, 144, 0),             # rows of out that start anywhere
])
def test_exact_sums_of_many_tiles(counts, Nc, Kd, cap, gather):
    check_exact(problem(counts, Nc, Kd, Nc + cap + 1, True, x_rows=500 if gather else None, cap=cap,
                        layout=MASKED if cap else CONTIG))
    if not gather:
        check_near(problem(counts, Nc, Kd, Nc + cap + 2, False, cap=cap, layout=MASKED if cap else CONTIG), BF)


@pytest.mark.parametrize("gather", [False, True])
def test_exact_sums_of_many_units_of_one_block(gather):
    """Several units a CTA, each over before the stages of the next are handed on."""
    check_exact(problem([5, 0, 9, 1] * 50, 2100, 128, 15, True, x_rows=31 if gather else None))
    check_exact(problem([3] * 100, 2100, 208, 16, True, x_rows=31 if gather else None))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("counts,Nc,Kd", [([2, 0, 1], 130, 272), ([300, 40], 392, 1168),
                                          ([20] * 9, 257, 784), ([1], 64, 7168), ([70, 700], 264, 2064)])
def test_codes_over_the_whole_range(counts, Nc, Kd, out):
    check_near(problem(counts, Nc, Kd, Nc, False), out)
    check_near(problem(counts, Nc, Kd, Nc + 1, False, x_rows=91), out)


def test_rows_that_read_nothing_are_zeros():
    for counts in ([4, 3], [130, 200]):
        p = problem(counts, 72, 144, 3, True, x_rows=9)
        p["src"][1], p["src"][4], p["src"][-1] = -1, 9, 1 << 30
        p["x"][0] = 0x7f  # what an invalid row must not read in its place
        p["src"][p["src"] == 0] = 1
        check_exact(p)
    p = problem([3, 2], 40, 64, 4, True, x_rows=5)
    p["x"], p["xs"] = p["x"][:0], p["xs"][:0]
    assert (run(p) == 0).all()


def test_scales_that_start_on_four_bytes():
    p = problem([70, 140], 136, 1024, 14, True)
    for name in ("xs", "ws"):
        t = p[name]
        p[name] = torch.cat([torch.zeros(1), t.flatten()]).cuda()[1:].view(t.shape)
    got = run(p).double().cpu().numpy()
    p["xs"], p["ws"] = p["xs"].cpu(), p["ws"].cpu()
    want, _, _ = want_of(p)
    np.testing.assert_array_equal(got, want)


def test_fewer_sources_than_rows():
    """Rows past the end of row_src read nothing (the masked layout's overlap of offsets)."""
    p = problem([4, 6], 64, 128, 5, True, x_rows=7, cap=8, layout=MASKED)
    full = run(p)
    p["src"] = p["src"][:7]
    cut = run(p)
    assert torch.equal(cut[:4], full[:4]) and torch.equal(cut[8:11], full[8:11])
    assert (cut[11:14] == 0).all() and (cut[4:8] == -77.0).all()


def test_nan_reaches_its_row_or_channel_alone():
    p = problem([3, 150], 136, 272, 6, True)
    p["x"][1, 130] = 0x7f
    p["w"][1, 130, 3] = 0xff
    got = run(p).cpu()
    nan = torch.isnan(got)
    want = torch.zeros_like(nan)
    want[1] = True
    want[3:, 130] = True
    assert torch.equal(nan, want)


def test_scales_of_zero_infinity_and_nan():
    p = problem([5, 140], 130, 256, 7, True)
    p["xs"][2, 1] = 0.0
    p["ws"][0, 1, 0] = 0.0
    check_exact(p)
    p["xs"][3, 0] = float("nan")
    p["ws"][1, 1, 1] = float("inf")
    got = run(p).cpu()
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[5:, 128:]).any()
    assert torch.isfinite(got[:3]).all() and torch.isfinite(got[4:, :128]).all()


def test_one_row_is_the_same_in_every_company():
    """A row's products do not depend on what else is in the call's tile: exact sums,
    alone, with others of its expert and among many experts."""
    p = problem([1], 200, 656, 8, True)
    alone = run(p)
    for n in (2, 33, 129, 400):
        q = dict(p, x=p["x"].expand(n, -1).contiguous(), xs=p["xs"].expand(n, -1).contiguous(), rows=n,
                 offs=torch.tensor([0, n], dtype=torch.int32))
        assert (run(q) == alone).all()


def test_offsets_that_break_their_order_stay_in_bounds():
    p = problem([6, 6, 6], 64, 128, 9, True)
    out = torch.full((18, 64), -77.0, device="cuda")
    for bad in ([0, 12, 6, 18], [5, 5, 100, 200], [-7, 3, 2, 1 << 30], [18, 0, 0, 0]):
        p["offs"] = torch.tensor(bad, dtype=torch.int32)
        run(p, out=out)
    torch.cuda.synchronize()


def test_second_stream_and_graph():
    p = problem([30, 0, 170], 264, 528, 10, True)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    out = torch.empty((200, 264), device="cuda")

    def call(stream=None):
        ep.ep_expert_matmul_fp8(d["x"], d["xs"], d["w"], d["ws"], d["offs"], out=out, stream=stream)
    want = run(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    # other rows per expert at replay: nothing of the capture's counts is kept
    d["offs"].copy_(torch.tensor([0, 150, 160, 200], dtype=torch.int32))
    p["offs"] = d["offs"].cpu()
    out.fill_(-1.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run(p))


def test_calls_that_run_together_on_two_streams():
    ps = [problem([64, 200, 3], 264, 1040, s, True) for s in (11, 12)]
    want = [run(p) for p in ps]
    ds = [{k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in p.items()} for p in ps]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, o, s in zip(ds, outs, streams):
            ep.ep_expert_matmul_fp8(d["x"], d["xs"], d["w"], d["ws"], d["offs"], out=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_output_of_unaligned_rows_and_odd_channels():
    for Nc in (1, 7, 33, 129, 255, 1023):
        check_exact(problem([2, 140], Nc, 144, Nc, True))
        check_near(problem([2, 140], Nc, 144, Nc, False), BF)


def test_weights_past_32_bits():
    """The last expert's weights start past 2^32 bytes."""
    E, Nc, Kd = 18, 4096, 65536
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free memory")
    g = torch.Generator().manual_seed(13)
    last, x = small_codes((Nc, Kd), g), small_codes((3, Kd), g)
    w = torch.zeros((E, Nc, Kd), dtype=torch.uint8, device="cuda")
    w[-1] = last.cuda()
    xs, ws = torch.ones((3, 512), device="cuda"), torch.ones((E, 32, 512), device="cuda")
    offs = torch.tensor([0] * E + [3], dtype=torch.int32, device="cuda")
    got = ep.ep_expert_matmul_fp8(x.cuda(), xs, w, ws, offs, out_dtype=F32).double()
    v = lambda t: torch.from_numpy(ref.e4m3(t.numpy()))  # noqa: E731
    want = v(x).float().cuda() @ v(last).float().cuda().T  # integers below 2^24: exact
    assert torch.equal(got, want.double())
