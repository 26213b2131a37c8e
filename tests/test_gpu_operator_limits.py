"""The modified-score and int8 entry points at the ends of what they document: caps of every size, tables whose entries
before the first visible key are gone, infinities and overflow in V, rows past n_rows, the widest tables."""
import numpy as np
import pytest
import test_gpu_score_mod as M
import torch

from oracle import score_mod as O
from paged_kv_cache_433_b200 import kvpaged as K

pytestmark = pytest.mark.gpu

# the kernels of paged_prefill_attention_mod: one softmax reference (bf16, cap <= 50), general tcgen05, warp MMA
PREFILL = [("bf16", 128, None), ("fp16", 128, None), ("bf16", 128, K.KV_DECODE_KERNEL_MMA), ("fp16", 64, None)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_433_b200 import build

    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _with_kernel(kernel, run):
    if kernel is not None:
        K.paged_decode_set_kernel(kernel)
    try:
        return run()
    finally:
        K.paged_decode_set_kernel(K.KV_DECODE_KERNEL_AUTO)


# ------------------------------------------------------------------ caps
CAPS = [1e-30, 1e-3, 600.0, 1e4, 1e10, 1e13, 1e14, 1e15, 1e20, 1e30, 1e36, 2.9e38, float(np.finfo(np.float32).max)]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype,Dh,P", [("bf16", 128, 16), ("fp16", 64, 32)])
def test_decode_mod_caps_of_every_size(dtype, Dh, P, cap):
    lens = [300, 1, 70]
    c = M._cache(lens, 2, Dh, P, dtype, seed=1)
    q = (2 * torch.randn((3, 8, Dh), generator=c["g"], device="cuda")).to(M.DT[dtype])
    ref, top = M._reference(c, q, np.arange(3), np.array(lens) - 1, Dh**-0.5, cap)
    for S in (1, 0):
        M._close(M._decode(c, q, Dh**-0.5, S, softcap=cap), ref, top, f"cap {cap}")


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype,Dh,kernel", PREFILL)
def test_prefill_mod_caps_of_every_size(dtype, Dh, kernel, cap):
    lens, chunks = [300, 90], np.array([40, 90])
    c = M._cache(lens, 2, Dh, 16, dtype, seed=2)
    b, pos, _ = M._rows(lens, chunks)
    q = (2 * torch.randn((len(b), 8, Dh), generator=c["g"], device="cuda")).to(M.DT[dtype])
    ref, top = M._reference(c, q, b, pos, Dh**-0.5, cap)
    got = _with_kernel(kernel, lambda: M._prefill(c, q, chunks, Dh**-0.5, softcap=cap))
    M._close(got, ref, top, f"cap {cap}")


@pytest.mark.parametrize("cap", [700.0, 1e5, 1e16])
@pytest.mark.parametrize("scale", [128**-0.5, 1e-6, 2e3])
def test_decode_mod_scores_below_at_and_above_a_large_cap(cap, scale):
    """Products of one, two, ... steps of a size, over the whole rise of the tanh: with slopes that hold the cap's multiples
    against one another every key keeps a weight, so that each capped score shows. A score of size s in log2 units errs by
    2^-21 s (a few roundings of 2^-24 and 2^-23), a weight by that times log 2, and so the row's sum over |v| <= top."""
    n, Dh = 12, 128
    c = M._cache([n], 1, Dh, 16, "bf16", seed=3)
    size = 2.0 ** np.round(np.log2(0.25 * cap / scale))  # the products k * size, k = 1 .. n, are exact
    c["kp"][int(c["tab"][0, 0]), 0] = 0
    c["kp"][int(c["tab"][0, 0]), 0, :n, 0] = torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * float(2.0 ** (np.log2(size) // 2))
    q = torch.zeros((1, 1, Dh), device="cuda", dtype=torch.bfloat16)
    q[0, 0, 0] = float(size / 2.0 ** (np.log2(size) // 2))
    s = cap * np.tanh(np.arange(1, n + 1) * size * scale / cap)
    # the last keys of the rise are level; the slope brings key 3 up to key 8
    slope = -(s[7] - s[2]) / 5
    ref, top = M._reference(c, q, np.zeros(1, int), np.array([n - 1]), scale, cap, torch.tensor([slope], dtype=torch.float32))
    got = M._decode(c, q, scale, 1, softcap=cap, alibi_slopes=torch.tensor([slope], dtype=torch.float32, device="cuda"))
    if 2.0**-21 * 1.45 * cap < 0.5:
        assert np.abs(got - ref).max() <= (2.0**-13 + 2.0**-21 * 1.45 * (cap + 11 * abs(slope))) * top.max()
    else:  # scores so far apart that one key has the whole weight
        assert np.isfinite(got).all()


# ------------------------------------------------------------------ pages behind a window are gone
@pytest.mark.parametrize("gone", [-1, 10**6])
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("dtype,Dh,kernel,mod", [
    ("bf16", 128, None, dict(softcap=30.0)), ("bf16", 128, None, dict()), ("fp16", 128, None, dict(softcap=30.0)),
    ("bf16", 128, K.KV_DECODE_KERNEL_MMA, dict()), ("fp16", 64, None, dict())], ids=str)
def test_prefill_mod_skips_pages_before_the_window(dtype, Dh, kernel, mod, P, gone):
    """Table entries of pages that no row of a chunk sees may be anything, and are no error."""
    lens, chunks = [700, 333, 90, 1000], np.array([100, 1, 90, 33])
    c = M._cache(lens, 2, Dh, P, dtype, seed=6)
    b, pos, start = M._rows(lens, chunks)
    q = torch.randn((len(b), 8, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    ks = np.where(b == 3, 970, 0)  # a document that begins inside the last chunk's window
    ref, top = M._reference(c, q, b, pos, Dh**-0.5, mod.get("softcap", 0.0), None, 75, ks)
    for i in range(4):
        first = max(0, lens[i] - chunks[i] - 75 + 1, 970 if i == 3 else 0)
        c["tab"][i, :first // P] = gone
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _with_kernel(kernel, lambda: M._prefill(c, q, chunks, Dh**-0.5, ks, err=err, window=75, **mod))
    M._close(got, ref, top, "pages gone")
    assert int(err) == 0
    c["tab"][3, -1] = gone  # one that is seen is reported
    _with_kernel(kernel, lambda: M._prefill(c, q, chunks, Dh**-0.5, ks, err=err, window=75, **mod))
    assert int(err) == K.KV_DEV_ERR_PAGE_RANGE


# ------------------------------------------------------------------ finite values that overflow
@pytest.mark.parametrize("kernel", [None, K.KV_DECODE_KERNEL_MMA])
@pytest.mark.parametrize("size,cap", [(1e30, 50.0), (3.3e38, 50.0), (3.3e38, 60.0), (3.3e38, 0.0)])
def test_prefill_mod_finite_values_that_overflow(size, cap, kernel):
    """Finite values whose weighted sum leaves fp32 give an infinity or not a number, never another finite value."""
    c = M._cache([300], 1, 128, 16, "bf16", seed=5)
    c["kp"] = c["kp"].abs()
    c["vp"].fill_(size)
    q = (500 * torch.randn((40, 4, 128), generator=c["g"], device="cuda").abs()).to(torch.bfloat16)
    got = _with_kernel(kernel, lambda: M._prefill(c, q, np.array([40]), 128**-0.5, softcap=cap))
    fine = np.isfinite(got)
    assert (np.abs(got[fine] / size - 1) < 2.0**-7).all()


@pytest.mark.parametrize("num_splits", [1, 0, 3])
def test_decode_mod_finite_values_that_overflow(num_splits):
    c = M._cache([2000], 1, 128, 16, "bf16", seed=5)
    q = (2 * torch.randn((1, 8, 128), generator=c["g"], device="cuda")).to(torch.bfloat16)
    c["vp"].copy_(3.3e38 * torch.sign(c["vp"].float()))
    got = M._decode(c, q, 128**-0.5, num_splits)
    ref, _ = M._reference(c, q, np.zeros(1, int), np.array([1999]), 128**-0.5)
    fine = np.isfinite(got)
    assert (np.abs(got - ref)[fine] < 2.0**-12 * 3.3e38).all()


# ------------------------------------------------------------------ infinities
@pytest.mark.parametrize("num_splits", [1, 2, 0])
def test_decode_mod_infinity_of_a_vanishing_weight(num_splits):
    """An infinity among the visible values gives its sign, however small its weight beside another piece's is."""
    lens = [600, 4000]
    c = M._cache(lens, 1, 128, 16, "bf16", seed=4)
    q = torch.randn((2, 4, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    for b, L in enumerate(lens):
        M._put(c, b, L - 3, None, 60 * torch.sign(q[b, 0].float()).to(torch.bfloat16), ("kp",))
        page, off = int(c["tab"][b, 0]), 5
        c["vp"][page, 0, off, 7] = float("-inf")
    q[:, 1:] = q[:, :1]
    ref, top = M._reference(c, q, np.arange(2), np.array(lens) - 1, 128**-0.5)
    assert (ref[:, :, 7] == -np.inf).all() and np.isfinite(np.delete(ref, 7, 2)).all()
    M._close(M._decode(c, q, 128**-0.5, num_splits), ref, top, "infinity")


@pytest.mark.parametrize("num_splits", [1, 0])
def test_decode_mod_infinity_in_a_long_row(num_splits):
    """The search for what made a sum NaN does not hold up the waits of the same CTA, however long the row is."""
    lens = [200000, 40, 90000]
    c = M._cache(lens, 1, 128, 16, "bf16", seed=9)
    q = torch.randn((3, 8, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    for b, t, d, what in ((0, 5, 3, "inf"), (0, 199999, 127, "-inf"), (2, 45000, 64, "nan"), (2, 89000, 65, "inf")):
        c["vp"][int(c["tab"][b, t // 16]), 0, t % 16, d] = float(what)
    ref, top = M._reference(c, q, np.arange(3), np.array(lens) - 1, 128**-0.5, 30.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    M._close(M._decode(c, q, 128**-0.5, num_splits, err=err, softcap=30.0), ref, top, "long row")
    assert int(err) == 0


@pytest.mark.parametrize("dtype,Dh,kernel", PREFILL)
def test_prefill_mod_infinities_in_many_tiles(dtype, Dh, kernel):
    """Infinities that some tiles of one sequence see, in stages that all of a tile's rows see and in such that only some do:
    every other row keeps its bits, those that see them say so, and no wait runs out, with many tiles a CTA and a long
    context."""
    lens, chunks = [70000, 9000, 12000], np.array([1400, 3000, 2500])
    H_kv, g = 4, 4
    c = M._cache(lens, H_kv, Dh, 16, dtype, seed=10)
    b, pos, start = M._rows(lens, chunks)
    q = torch.randn((len(b), H_kv * g, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    mod = dict(softcap=20.0)
    ks = np.maximum(0, np.where(b == 2, pos - 2000, 0))
    run = lambda err=None: _with_kernel(kernel, lambda: M._prefill(c, q, chunks, Dh**-0.5, ks, err=err, **mod))  # noqa: E731
    clean = run()
    marks = [(0, 69000, 1, 5, "inf"), (0, 3, 2, 6, "-inf"), (0, 69001, 0, 7, "nan"), (2, 10500, 3, 8, "inf"), (2, 11999, 3, 9, "inf")]
    for i, t, h, d, what in marks:
        c["vp"][int(c["tab"][i, t // 16]), h, t % 16, d] = float(what)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(err)
    assert int(err) == 0
    want = clean.copy()
    touched = np.zeros((len(b), H_kv * g), bool)
    for i, t, h, d, what in marks:
        sees = (b == i) & (pos >= t) & (ks <= t)
        want[sees, h * g:(h + 1) * g, d] = float(what)
        touched[sees, h * g:(h + 1) * g] = True
    special = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[special & ~np.isnan(want)], want[special & ~np.isnan(want)])
    # the other dims of a row that sees one: the same but for the order of its sums
    assert np.array_equal(got[~touched], clean[~touched])
    other = touched[:, :, None] & ~special
    assert np.abs(got[other] - clean[other]).max() <= 2.0**-13 * 6


# ------------------------------------------------------------------ rows past n_rows
@pytest.mark.parametrize("dtype,Dh,kernel", PREFILL)
@pytest.mark.parametrize("n_rows,starts", [(10, [0, 40]), (33, [0, 30, 70]), (64, [0, 64, 90]), (50, [0, 5, 5, 49, 120])])
def test_prefill_mod_rows_past_n_rows_are_left_alone(dtype, Dh, kernel, n_rows, starts):
    """Chunks that reach past n_rows: their rows before it are computed, those past it not written."""
    chunks = np.diff(starts)
    lens = chunks + 100
    c = M._cache(lens, 2, Dh, 16, dtype, seed=7)
    b, pos, _ = M._rows(lens, chunks)
    q = torch.randn((starts[-1], 8, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    ref, top = M._reference(c, q, b, pos, Dh**-0.5, 20.0, None, 64)
    out = torch.full(q.shape, 7.0, device="cuda")  # (as large as the chunks: what a fault would write stays inside)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d_start, tab, d_len = M._d(starts), torch.from_numpy(c["tab"]).cuda(), M._d(lens)
    _with_kernel(kernel, lambda: K.paged_prefill_attention_mod(
        out[:n_rows], q[:n_rows], d_start, int(chunks.max()), c["kp"], c["vp"], tab, d_len, Dh**-0.5, softcap=20.0, window=64,
        err_flag=err))
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert (got[n_rows:] == 7).all()
    M._close(got[:n_rows], ref[:n_rows], top[:n_rows], "rows before n_rows")


@pytest.mark.parametrize("dtype,Dh,kernel", PREFILL)
def test_prefill_mod_rows_past_max_q_len_are_left_alone(dtype, Dh, kernel):
    lens, chunks = [200, 150, 90], np.array([70, 48, 90])
    c = M._cache(lens, 2, Dh, 16, dtype, seed=7)
    b, pos, start = M._rows(lens, chunks)
    q = torch.randn((len(b), 8, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    ref, top = M._reference(c, q, b, pos, Dh**-0.5, 20.0)
    out = torch.full(q.shape, 7.0, device="cuda")
    got = _with_kernel(kernel, lambda: M._prefill(c, q, chunks, Dh**-0.5, max_q_len=48, out=out, softcap=20.0))
    past = np.arange(len(b)) - start[b] >= 48
    assert (got[past] == 7).all()
    M._close(got[~past], ref[~past], top[~past], "rows before max_q_len")


# ------------------------------------------------------------------ wide tables
def test_decode_mod_workspace_of_the_widest_tables():
    """paged_decode_ext_workspace_bytes holds for any window: also where the rows laid end to end leave 32 bits without a
    window and not with one."""
    B, H_kv, mb, P = 1024, 8, 262144, 16
    c = M._cache([900] * 3, H_kv, 64, P, "bf16", seed=8)
    tab = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    lens = np.zeros(B, int)
    rows = np.array([0, 511, 1023])
    lens[rows] = 900
    tab[torch.from_numpy(rows).cuda(), :c["tab"].shape[1]] = torch.from_numpy(c["tab"]).cuda()
    q = torch.randn((B, H_kv, 64), generator=c["g"], device="cuda").to(torch.bfloat16)
    out = torch.full(q.shape, float("nan"), device="cuda")
    ws = torch.empty(max(16, K.paged_decode_ext_workspace_bytes(B, H_kv, H_kv, 64, mb, P)), dtype=torch.uint8, device="cuda")
    K.paged_decode_attention_mod(out, q, c["kp"], c["vp"], tab, M._d(lens), 0.125, window=700, workspace=ws)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    ref, top = M._reference(c, q[torch.from_numpy(rows).cuda()], np.arange(3), np.full(3, 899), 0.125, 0.0, None, 700)
    M._close(got[rows], ref, top, "wide table")
    assert not np.delete(got, rows, 0).any()


# ------------------------------------------------------------------ one launch behind another
@pytest.mark.parametrize("graph", [False, True])
def test_int8_calls_behind_one_another_read_what_the_last_one_wrote(graph):
    """Norm + rotation into k_out, the append of it, a copy of its pages, the read-back and a decode whose rows are cut between
    CTAs, step after step over the same buffers with other values: every launch reads what the one before has just written,
    although it may have started before that one ended."""
    T, H_q, H_kv, Dh, P, n = 4096, 8, 2, 128, 16, 256
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.empty((T, H_kv, Dh), dtype=torch.bfloat16, device="cuda")
    v, k_out = torch.empty_like(x), torch.empty_like(x)
    cos_sin = torch.cat([torch.ones((4, Dh // 2)), torch.zeros((4, Dh // 2))], 1).cuda()  # no rotation
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros((2 * n, H_kv, P, Dh), dtype=torch.int8, device="cuda") for _ in range(2))
    sc = torch.zeros((2 * n, H_kv, 2, P), device="cuda")
    ko, vo = (torch.zeros((n, H_kv, P, Dh), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.arange(T, device="cuda")
    lo, hi = (torch.arange(i, i + n, dtype=torch.int32, device="cuda") for i in (0, n))
    tab = hi[None].contiguous()
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    q = torch.randn((1, H_q, Dh), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.zeros((1, H_q, Dh), device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")

    def step():
        K.kv_norm_rope_append(None, None, x, None, None, pos, cos_sin, None, 1e-6, P, k_out=k_out)
        K.kv_append_int8(kp, vp, sc, k_out, v, slots, P)
        K.kv_copy_pages_int8(kp, vp, sc, lo, hi)
        K.kv_dequant_pages_int8(ko, vo, kp, vp, sc, hi, lo)
        K.paged_decode_attention_int8(out, q, kp, vp, sc, tab, lens, Dh**-0.5, workspace=ws)

    x.normal_(generator=g), v.normal_(generator=g)
    step()
    torch.cuda.synchronize()
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
            step()
    for i in range(20):
        x.normal_(generator=g), v.normal_(generator=g)
        v.mul_(2.0 ** (i % 5))
        if graph:
            cg.replay()
        else:
            step()
        torch.cuda.synchronize()
        rows = lambda t: t.transpose(1, 2).reshape(T, H_kv, Dh).float().cpu().numpy()  # noqa: E731
        for got, new in ((ko, k_out), (vo, v)):
            codes, scales = O.quantise_int8(new.float().cpu().numpy())
            want = torch.from_numpy(codes.astype(np.float32) * scales[..., None]).to(torch.bfloat16).float().numpy()
            assert np.array_equal(rows(got), want), f"step {i}"
        kd, vd = (rows(t.float()).astype(np.float64) for t in (ko, vo))
        ref = O.attend_row(q[0].double().cpu().numpy(), kd, vd, T - 1, T, Dh**-0.5)
        # the pages read back are rounded to bf16 (2^-9 of K and of V), their codes are not: scores up to 6 err by 6 * 2^-9
        assert np.abs(out[0].double().cpu().numpy() - ref).max() <= (2 * 6 * 2.0**-9 + 2.0**-9) * np.abs(vd).max(), f"step {i}"
