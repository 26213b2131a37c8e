"""Where the int8 cache's and the modified scores' kernels change their way of working: long accumulations, rows cut
into many pieces, batches beyond the balanced launch, one softmax reference at a cap's two ends, shared workspaces."""
import numpy as np
import pytest
import test_gpu_int8 as I8
import test_gpu_score_mod as M
import torch

from paged_kv_cache_433_b200 import kvpaged as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_433_b200 import build

    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _near(got, ref, what, bound=1e-5):
    """Of values with a mean of 1 nothing averages out. Weights and their residuals err by 2^-17 (7.6e-6) at most, both
    products' sums of 16 and the sums of weights by a few 2^-24: 1e-5 bounds their sum."""
    off = np.sqrt(((got - ref) ** 2).sum() / (ref**2).sum())
    assert off <= bound, f"{what}: {off:.2e} of the result"


def _mod_sums(lens, num_splits, H_q, H_kv, Dh, P, dtype, seed=1, **mod):
    c = M._cache(lens, H_kv, Dh, P, dtype, seed)
    c["vp"] += 1
    q = torch.randn((len(lens), H_q, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    ref, _ = M._reference(c, q, np.arange(len(lens)), np.asarray(lens) - 1, Dh**-0.5, mod.get("softcap", 0.0))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = M._decode(c, q, Dh**-0.5, num_splits, err=err, **mod)
    assert int(err) == 0
    return got, ref


@pytest.mark.parametrize("dtype,Dh,P,H_q,H_kv", [("bf16", 128, 16, 4, 1), ("fp16", 128, 32, 8, 1), ("bf16", 64, 16, 12, 1),
                                                 ("bf16", 128, 16, 48, 1)])
@pytest.mark.parametrize("num_splits", [1, 2])
def test_decode_mod_long_pieces(dtype, Dh, P, H_q, H_kv, num_splits):
    """A warp's output sums move out of the MMA accumulators several times within one piece."""
    got, ref = _mod_sums([40011, 3, 18000], num_splits, H_q, H_kv, Dh, P, dtype, softcap=30.0)
    _near(got, ref, "long pieces")


@pytest.mark.parametrize("dtype,Dh,P,H_q,H_kv", [("bf16", 128, 16, 4, 1), ("fp16", 128, 32, 8, 1), ("bf16", 64, 16, 12, 1)])
@pytest.mark.parametrize("num_splits", [1, 2])
def test_decode_int8_long_pieces(dtype, Dh, P, H_q, H_kv, num_splits):
    c = I8._decode_case([40011, 3, 18000], H_q, H_kv, Dh, P, dtype, seed=3)
    c["vp"].clamp_(min=0)  # values of one sign
    ref, _ = I8._reference(c)
    _near(I8._decode(c, num_splits), ref, "long pieces")


def test_decode_balanced_pieces_longer_than_an_accumulation():
    """Balanced launch with so many tokens that a CTA's pieces pass 4 x 2048 keys, several pieces to a CTA: the same
    lengths in rows that share their pages."""
    P, H_q, H_kv, Dh, B = 16, 32, 8, 128, 130
    lens = np.full(B, 9000)
    lens[::3] = 20011
    lens[5::9] = 40
    c = M._cache([20011], H_kv, Dh, P, "bf16", 4)
    c["vp"] += 1
    c["tab"], c["lens"] = np.repeat(c["tab"], B, 0), lens
    q = torch.randn((B, H_q, Dh), generator=c["g"], device="cuda").to(torch.bfloat16)
    got = M._decode(c, q, Dh**-0.5, 0, softcap=30.0)
    rows = np.array([0, 1, 5, 60, 129])
    ref, _ = M._reference(c, q[torch.from_numpy(rows).cuda()], rows, lens[rows] - 1, Dh**-0.5, 30.0)
    _near(got[rows], ref, "balanced")
    one = M._decode(c, q, Dh**-0.5, 1, softcap=30.0)  # one CTA per row: every row against another cut of the work
    _near(got, one, "balanced against whole rows", 2e-5)


@pytest.mark.parametrize("lens", [[30000], [25000, 0, 517], [17, 9000, 1, 6001]], ids=str)
@pytest.mark.parametrize("H_q,H_kv", [(8, 2), (16, 1), (5, 5)])
def test_decode_few_long_rows(lens, H_q, H_kv):
    """A small batch's rows are cut into dozens of pieces, merged row by row."""
    got, ref = _mod_sums(lens, 0, H_q, H_kv, 128, 16, "bf16")
    _near(got, ref, "modified")
    c = I8._decode_case(lens, H_q, H_kv, 128, 16, "bf16", seed=5)
    ref, top = I8._reference(c)
    I8._close(I8._decode(c), ref, top, "int8")


def test_decode_more_sequences_than_a_balanced_launch_takes():
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 400, 1100)
    lens[7] = 400
    rows = np.r_[0, 7, np.arange(3, 1100, 97), 1099]
    c = M._cache(lens, 1, 64, 16, "bf16", 6)
    q = torch.randn((1100, 4, 64), generator=c["g"], device="cuda").to(torch.bfloat16)
    for win in (0, 300):
        ref, top = M._reference(c, q[torch.from_numpy(rows).cuda()], rows, lens[rows] - 1, 0.125, 9.0, None, win)
        M._close(M._decode(c, q, 0.125, 0, softcap=9.0, window=win)[rows], ref, top, f"window {win}")
    c = I8._decode_case(lens, 4, 1, 64, 16, "fp16", seed=6)
    ref, top = I8._reference(c, rows.tolist())
    I8._close(I8._decode(c)[rows], ref[rows], top[rows], "int8")


@pytest.mark.parametrize("B,mb", [(3, 2000), (300, 100)])
def test_decode_all_rows_empty(B, mb):
    c = M._cache([16], 2, 128, 16, "bf16", 7)
    c["tab"], c["lens"] = np.full((B, mb), -1, np.int32), np.zeros(B, int)
    q = torch.randn((B, 8, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    assert not M._decode(c, q, 0.1, 0, softcap=5.0).any()
    # every row's first visible key lies behind its length
    c["tab"][:] = 0
    c["lens"][:] = 16
    assert not M._decode(c, q, 0.1, 0, key_start=np.full(B, 10**9), softcap=5.0).any()


@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("dtype,Dh,kernel,mod", [
    ("bf16", 128, None, dict(softcap=30.0)), ("bf16", 128, None, dict(softcap=60.0)), ("fp16", 128, None, dict(softcap=30.0)),
    ("bf16", 128, K.KV_DECODE_KERNEL_MMA, dict(softcap=30.0)), ("fp16", 64, None, dict()), ("bf16", 64, None, dict())], ids=str)
def test_prefill_mod_long_sums(dtype, Dh, kernel, mod, P):
    """Tiles of 64 and of 128 rows over contexts longer than one accumulation."""
    lens, chunks = [9000, 6333], np.array([150, 33])
    c = M._cache(lens, 2, Dh, P, dtype, seed=8)
    c["vp"] += 1
    b, pos, _ = M._rows(lens, chunks)
    q = torch.randn((len(b), 8, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    rows = np.r_[0, 15, 16, 149, 150, 182]
    ref, _ = M._reference(c, q[torch.from_numpy(rows).cuda()], b[rows], pos[rows], Dh**-0.5, mod.get("softcap", 0.0))
    if kernel is not None:
        K.paged_decode_set_kernel(kernel)
    try:
        got = M._prefill(c, q, chunks, Dh**-0.5, **mod)
    finally:
        K.paged_decode_set_kernel(K.KV_DECODE_KERNEL_AUTO)
    # An accumulation of 2048 keys is 128 steps of 16, each the product with the weights and that with their residuals
    # added to it and rounded towards zero: 256 losses of less than 2^-23 of a sum that only grows.
    _near(got[rows], ref, "long sums", 1e-5 + 256 * 2.0**-23)


@pytest.mark.parametrize("v_size", [1e-6, 1.0, 1e15])
@pytest.mark.parametrize("sign", [1, -1])
def test_prefill_mod_scores_at_the_cap(sign, v_size):
    """Every score of some heads at +-50, the largest cap that takes one softmax reference for all rows."""
    lens, chunks = [200, 70], np.array([64, 70])
    c = M._cache(lens, 2, 128, 16, "bf16", seed=9)
    c["kp"] = c["kp"].abs()  # (a NaN stays one)
    c["vp"] = ((c["vp"].float() + 1) * v_size).to(torch.bfloat16)
    b, pos, _ = M._rows(lens, chunks)
    q = torch.randn((len(b), 8, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    q[:, ::2] = sign * 500 * q[:, ::2].abs()
    ref, _ = M._reference(c, q, b, pos, 128**-0.5, 50.0)
    got = M._prefill(c, q, chunks, 128**-0.5, softcap=50.0)
    assert np.isfinite(got).all()
    _near(got, ref, "cap", 1e-5 + 256 * 2.0**-23)  # a chunk: see test_prefill_mod_long_sums


def test_graphs_that_share_a_workspace_and_side_streams():
    """Two captured graphs and eager calls of both decode kernels use one workspace in turn, on streams other than the
    tensors' own: nothing in it is kept from call to call."""
    lens = [5000, 0, 700, 64]
    cm = M._cache(lens, 2, 128, 16, "bf16", 10)
    q = torch.randn((4, 8, 128), generator=cm["g"], device="cuda").to(torch.bfloat16)
    ci = I8._decode_case(lens, 16, 4, 128, 16, "bf16", seed=10)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    d_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    tm, ti = (torch.from_numpy(c["tab"]).cuda() for c in (cm, ci))
    om, oi = torch.empty((4, 8, 128), device="cuda"), torch.empty((4, 16, 128), device="cuda")
    run_m = lambda: K.paged_decode_attention_mod(om, q, cm["kp"], cm["vp"], tm, d_len, 0.09, softcap=20.0, workspace=ws)  # noqa: E731
    run_i = lambda: K.paged_decode_attention_int8(oi, ci["q"], ci["kp"], ci["vp"], ci["sc"], ti, d_len, 0.09, workspace=ws)  # noqa: E731
    run_m(), run_i()
    torch.cuda.synchronize()
    want_m, want_i = om.clone(), oi.clone()
    ref, top = M._reference(cm, q, np.arange(4), np.array(lens) - 1, 0.09, 20.0)
    M._close(want_m.double().cpu().numpy(), ref, top, "eager")
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for run in (run_m, run_i):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run()
            run()
        graphs.append(g)
    for k in range(6):
        om.fill_(float("nan")), oi.fill_(float("nan"))
        if k % 2:
            d_len.fill_(33)  # other work in between
            graphs[0].replay(), graphs[1].replay()
            d_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graphs[k % 2].replay()
        graphs[1 - k % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(om, want_m) and torch.equal(oi, want_i)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            om.fill_(float("nan"))
            run_m()
        side.synchronize()
        assert torch.equal(om, want_m)


@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("mod", [dict(softcap=20.0), dict(softcap=50.0, window=200, docs=True), dict(softcap=3.0, window=1),
                                 dict(softcap=30.0, prefix=True)], ids=str)
def test_prefill_mod_capped_many_tiles(mod, P):
    """Tiles of very different cost, some without rows or visible keys, a chunk longer than its sequence, in a launch that
    CTAs share out among themselves: eager, on two streams at once, and replayed."""
    rng = np.random.default_rng(P)
    B = 48
    chunks = rng.integers(0, 260, B)
    chunks[[2, 11]] = 0
    lens = chunks + (rng.integers(0, 1500, B) * (rng.random(B) < 0.6)).astype(int)
    lens[20], chunks[20] = 30, 40  # refused
    c = M._cache(lens, 8, 128, P, "bf16", seed=P)
    b, pos, start = M._rows(lens, chunks)
    q = torch.randn((len(b) + 9, 16, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    ks = None
    if mod.get("docs"):
        ks = np.r_[np.maximum(0, pos - rng.integers(0, 300, len(pos))), np.zeros(9, int)]
        ks[start[5]:start[6]] = 10**6  # a sequence whose rows see nothing
    prefix = rng.integers(-5, 700, B) if mod.get("prefix") else None
    cap, win = mod["softcap"], mod.get("window", 0)
    out = torch.full(q.shape, 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(key_start=ks, prefix=prefix, max_q_len=300, softcap=cap, window=win)
    got = M._prefill(c, q, chunks, 0.09, err=err, out=out, **args)
    assert int(err) == K.KV_DEV_ERR_SEQ_LEN
    assert (got[len(b):] == 7).all() and not got[start[20]:start[21]].any()
    rows = np.unique(np.r_[start[:-1], start[1:] - 1, rng.integers(0, len(b), 60)].clip(0, len(b) - 1))
    rows = rows[b[rows] != 20]
    ref, top = M._reference(c, q[torch.from_numpy(rows).cuda()], b[rows], pos[rows], 0.09, cap, None, win,
                            None if ks is None else ks[rows], prefix)
    M._close(got[rows], ref, top, str(mod))
    want = out.clone()
    d = dict(start=M._d(start), tab=torch.from_numpy(c["tab"]).cuda(), lens=M._d(lens), ks=M._d(ks), pf=M._d(prefix))

    def run(o):
        K.paged_prefill_attention_mod(o, q, d["start"], 300, c["kp"], c["vp"], d["tab"], d["lens"], 0.09, softcap=cap,
                                      window=win, key_start=d["ks"], prefix_lens=d["pf"])

    outs, streams = [torch.full(q.shape, 7.0, device="cuda") for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o, s in zip(outs, streams):
            with torch.cuda.stream(s):
                run(o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[0])
        run(outs[1])
    for o in outs:
        o.fill_(7.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("mod", [dict(softcap=20.0), dict(softcap=2.0, alibi=True), dict(window=50), dict()], ids=str)
@pytest.mark.parametrize("dtype,Dh,kernel", [("bf16", 128, None), ("fp16", 128, None), ("fp16", 64, None),
                                             ("bf16", 128, K.KV_DECODE_KERNEL_MMA)])
def test_prefill_mod_hidden_keys_have_no_effect(dtype, Dh, kernel, mod):
    """Not one bit of a row changes with the keys behind it, in its own tile or in the unused part of a page."""
    lens, chunks = [301, 90], np.array([150, 90])
    c = M._cache(lens, 2, Dh, 16, dtype, seed=21)
    b, pos, start = M._rows(lens, chunks)
    q = torch.randn((len(b), 8, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    mod = dict(mod, alibi_slopes=M._slopes(8)) if mod.get("alibi") else mod
    mod = {k: v for k, v in mod.items() if k != "alibi"}
    if kernel is not None:
        K.paged_decode_set_kernel(kernel)
    try:
        first = M._prefill(c, q, chunks, Dh**-0.5, **mod)
        for s, t0 in ((0, 270), (1, 33)):
            for t in range(t0, lens[s]):
                M._put(c, s, t, None, 40.0 if t % 2 else -300.0)
        for p in ("kp", "vp"):
            c[p].nan_to_num_(nan=77.0)
        again = M._prefill(c, q, chunks, Dh**-0.5, **mod)
    finally:
        K.paged_decode_set_kernel(K.KV_DECODE_KERNEL_AUTO)
    same = np.where(b == 0, pos < 270, pos < 33)
    assert np.array_equal(first[same], again[same]) and not np.array_equal(first, again)


@pytest.mark.parametrize("num_splits", [0, 1])
@pytest.mark.parametrize("mod", [dict(softcap=20.0), dict(softcap=2.0), dict(window=50)], ids=str)
def test_decode_mod_hidden_keys_have_no_effect(mod, num_splits):
    lens = [301, 90, 5]
    c = M._cache(lens, 2, 128, 32, "bf16", seed=22)
    q = torch.randn((3, 8, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    first = M._decode(c, q, 128**-0.5, num_splits, key_start=[3, 44, 2], **mod)
    for p in ("kp", "vp"):
        c[p].nan_to_num_(nan=500.0)
    for s, t1 in ((0, 3), (1, 44), (2, 2)):
        for t in range(t1):
            M._put(c, s, t, None, 300.0)
    assert np.array_equal(first, M._decode(c, q, 128**-0.5, num_splits, key_start=[3, 44, 2], **mod))


@pytest.mark.parametrize("B", [1, 33, 200])
@pytest.mark.parametrize("dtype,Dh,H_q,H_kv,mod", [("bf16", 128, 8, 2, dict(softcap=30.0)), ("fp16", 128, 8, 8, dict(window=70)),
                                                   ("bf16", 64, 12, 4, dict(softcap=4.0)), ("bf16", 128, 64, 1, dict(softcap=9.0))])
def test_prefill_mod_one_long_chunk_among_short_ones(dtype, Dh, H_q, H_kv, mod, B):
    """Tiles lie behind one another whatever the chunks' lengths are: one long chunk, chunks of one token, empty ones."""
    rng = np.random.default_rng(B)
    chunks = rng.integers(0, 3, B)
    chunks[B // 3] = 401
    lens = chunks + rng.integers(0, 90, B)
    c = M._cache(lens, H_kv, Dh, 16, dtype, seed=B)
    b, pos, start = M._rows(lens, chunks)
    q = torch.randn((len(b), H_q, Dh), generator=c["g"], device="cuda").to(M.DT[dtype])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = M._prefill(c, q, chunks, Dh**-0.5, err=err, **mod)
    assert int(err) == 0 and np.isfinite(got).all()
    rows = np.unique(np.r_[0, len(b) - 1, start[B // 3], start[B // 3 + 1] - 1, rng.integers(0, len(b), 40)])
    ref, top = M._reference(c, q[torch.from_numpy(rows).cuda()], b[rows], pos[rows], Dh**-0.5, mod.get("softcap", 0.0), None,
                            mod.get("window", 0))
    M._close(got[rows], ref, top, "mixed chunks")
