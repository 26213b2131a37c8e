"""GPU parity of paged_decode_attention_mod and paged_prefill_attention_mod (tanh cap, distance bias, sliding window,
documents, bidirectional prefix) against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import score_mod as O
from paged_kv_cache_433_b200 import kvpaged as K

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_433_b200 import build

    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _cache(lens, H_kv, Dh, P, dtype, seed):
    """Random K/V of each sequence in randomly placed pages; every unused slot holds NaN, unused table entries -1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = np.asarray(lens)
    need = -(-lens // P)
    mb = max(1, int(need.max()))
    num_pages = int(need.sum()) + 2
    kp = torch.randn((num_pages, H_kv, P, Dh), generator=g, device="cuda").to(DT[dtype])
    vp = torch.randn((num_pages, H_kv, P, Dh), generator=g, device="cuda").to(DT[dtype])
    order = torch.randperm(num_pages, generator=g, device="cuda").cpu().numpy()
    tab = np.full((len(lens), mb), -1, np.int32)
    used = np.zeros((num_pages, P), bool)
    at = 0
    for b, L in enumerate(lens):
        tab[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = np.arange(L)
        used[tab[b][t // P], t % P] = True
    hole = torch.from_numpy(~used).cuda()[:, None, :, None]
    kp.masked_fill_(hole, float("nan"))
    vp.masked_fill_(hole, float("nan"))
    return dict(lens=lens, tab=tab, kp=kp, vp=vp, P=P, H_kv=H_kv, Dh=Dh, dtype=dtype, g=g)


def _put(c, b, t, head, what, pools=("kp", "vp")):
    """K and V of token t of sequence b (one head, or all)."""
    page, off = int(c["tab"][b, t // c["P"]]), t % c["P"]
    for p in pools:
        c[p][page, head if head is not None else slice(None), off] = what


def _rows(lens, chunks):
    b = np.repeat(np.arange(len(chunks)), chunks)
    start = np.concatenate([[0], np.cumsum(chunks)])
    return b, (np.asarray(lens) - chunks)[b] + np.arange(len(b)) - start[b], start


def _reference(c, q, b_of, pos, scale, softcap=0.0, slopes=None, window=0, key_start=None, prefix=None):
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    kp, vp, q = n(c["kp"]), n(c["vp"]), n(q)
    sl = None if slopes is None else n(slopes)
    out, top = np.zeros(q.shape), np.zeros((len(q), 1, 1))
    seqs = {b: tuple(O.gather(x, c["tab"][b], int(c["lens"][b]), c["P"]) for x in (kp, vp)) for b in set(b_of.tolist())}
    for r in range(len(q)):
        b = int(b_of[r])
        k, v = seqs[b]
        L = int(c["lens"][b])
        ks = None if key_start is None else key_start[r]
        pf = None if prefix is None else prefix[b]
        out[r] = O.attend_row(q[r], k, v, int(pos[r]), L, scale, softcap, sl, window, ks, pf)
        lo, hi = O.visible(int(pos[r]), L, window, ks, pf)
        top[r] = np.nanmax(np.abs(v[lo:hi][np.isfinite(v[lo:hi])]), initial=0) if lo < hi else 0
    return out, top


def _close(got, ref, top, what):
    """A probability enters the product as a 16-bit value and its residual (2^-14 of it where both are truncated), a
    score errs by a few 2^-22 of its size before the cap and 2^-22 of the cap behind it (both below 60 here), the sums
    by 2^-23 a step: 2^-13 of the largest visible |v| bounds their sum. Not-a-number and infinite outputs agree."""
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), what
    err = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)), 0)
    assert (err <= 2.0**-13 * top).all(), f"{what}: worst {np.max(err / np.maximum(top, 1e-30)):.2e} of max |v|"
    off, size = np.sqrt((err**2).sum()), np.sqrt((ref[fine] ** 2).sum())
    assert off <= 1e-5 * size or size == 0, f"{what}: {off / size:.2e} of the result"


def _slopes(H_q):
    return torch.exp2(-8.0 * torch.arange(1, H_q + 1, device="cuda") / H_q).float()


def _d(a):
    return None if a is None else torch.from_numpy(np.asarray(a, np.int32)).cuda()


# ------------------------------------------------------------------ decode
def _decode(c, q, scale, num_splits=0, key_start=None, err=None, **mod):
    B, H_q, Dh = q.shape
    out = torch.full((B, H_q, Dh), float("nan"), device="cuda")
    need = K.paged_decode_ext_workspace_bytes(B, H_q, c["H_kv"], Dh, c["tab"].shape[1], c["P"], num_splits)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    K.paged_decode_attention_mod(out, q, c["kp"], c["vp"], torch.from_numpy(c["tab"]).cuda(), _d(c["lens"]), scale,
                                 num_splits=num_splits, workspace=ws, err_flag=err, key_start=_d(key_start), **mod)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


MODS = [dict(), dict(softcap=5.0), dict(softcap=50.0, window=40), dict(alibi=True), dict(window=1), dict(window=17, docs=True),
        dict(softcap=20.0, alibi=True, docs=True), dict(docs=True), dict(window=10**9), dict(softcap=0.5, window=100)]
SHAPES = [("bf16", 128, 16, 32, 8), ("fp16", 128, 32, 8, 8), ("fp16", 64, 16, 12, 4), ("bf16", 64, 32, 32, 1),
          ("bf16", 128, 16, 64, 1), ("fp16", 128, 16, 28, 4)]


@pytest.mark.parametrize("mod", MODS, ids=str)
@pytest.mark.parametrize("dtype,Dh,P,H_q,H_kv", SHAPES)
def test_decode_mod(dtype, Dh, P, H_q, H_kv, mod):
    lens = [1, 0, P, 2 * P + 1, 300, 517, 200]
    c = _cache(lens, H_kv, Dh, P, dtype, seed=H_q + Dh)
    q = (2 * torch.randn((len(lens), H_q, Dh), generator=c["g"], device="cuda")).to(DT[dtype])
    ks = [0, 5, -3, P, 299, 250, 200] if mod.get("docs") else None  # 200 of 200: sees nothing
    sl = _slopes(H_q) if mod.get("alibi") else None
    cap, win = mod.get("softcap", 0.0), mod.get("window", 0)
    pos = np.asarray(lens) - 1
    scale = Dh**-0.5
    ref, top = _reference(c, q, np.arange(len(lens)), pos, scale, cap, sl, win, ks)
    for S in (1, 0, 3):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _decode(c, q, scale, S, ks, err, softcap=cap, alibi_slopes=sl, window=win)
        assert int(err) == 0
        _close(got, ref, top, f"S={S}")


@pytest.mark.parametrize("mod", [dict(softcap=30.0), dict(window=100), dict(docs=True, alibi=True)], ids=str)
def test_decode_mod_planned_many_rows(mod):
    rng = np.random.default_rng(7)
    lens = np.rint(np.exp(rng.normal(4.5, 1.0, 150))).astype(int).clip(0, 900)
    lens[3], lens[4] = 0, 880
    c = _cache(lens, 8, 128, 16, "bf16", seed=3)
    q = torch.randn((150, 32, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    ks = (lens * rng.random(150)).astype(int) if mod.get("docs") else None
    if ks is not None:
        ks[10] = lens[10] + 4
    sl = _slopes(32) if mod.get("alibi") else None
    got = _decode(c, q, 128**-0.5, 0, ks, softcap=mod.get("softcap", 0.0), alibi_slopes=sl, window=mod.get("window", 0))
    rows = np.r_[3, 4, 10, np.arange(0, 150, 11)]
    ref, top = _reference(c, q[torch.from_numpy(rows).cuda()], rows, lens[rows] - 1, 128**-0.5, mod.get("softcap", 0.0), sl,
                          mod.get("window", 0), None if ks is None else ks[rows])
    _close(got[rows], ref, top, "planned")


@pytest.mark.parametrize("num_splits", [1, 4])
def test_decode_mod_hidden_values_and_visible_nan(num_splits):
    """NaN and infinities before the first visible key have no effect; a visible NaN or infinity shows."""
    c = _cache([200, 200, 200, 200], 2, 128, 16, "bf16", seed=5)
    q = torch.randn((4, 8, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    for t in range(0, 150):
        _put(c, 0, t, None, float("nan") if t % 2 else float("inf"))
    _put(c, 1, 190, 1, float("nan"), ("kp",))
    _put(c, 2, 160, 0, float("inf"), ("vp",))
    _put(c, 3, 149, None, float("nan"))
    ref, top = _reference(c, q, np.arange(4), np.full(4, 199), 128**-0.5, 10.0, None, 50)
    _close(_decode(c, q, 128**-0.5, num_splits, softcap=10.0, window=50), ref, top, "hidden values")
    assert np.isnan(ref[1, 4:]).all() and np.isinf(ref[2, :4]).all() and np.isfinite(ref[[0, 3]]).all()


def test_decode_mod_skips_pages_before_the_window():
    """Pages that no visible key is on are not read: their table entries may be anything."""
    c = _cache([300, 90], 2, 128, 16, "fp16", seed=6)
    q = torch.randn((2, 8, 128), generator=c["g"], device="cuda").to(torch.float16)
    ref, top = _reference(c, q, np.arange(2), np.array([299, 89]), 128**-0.5, 0.0, None, 33)
    c["tab"][0, :(300 - 33) // 16] = 10**6
    c["tab"][1, :(90 - 33) // 16] = -1
    for S in (1, 0, 2):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        _close(_decode(c, q, 128**-0.5, S, err=err, window=33), ref, top, f"S={S}")
        assert int(err) == 0
    c["tab"][0, -1] = 10**6  # a visible page outside the pool is reported and skipped
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _decode(c, q, 128**-0.5, 1, err=err, window=33)
    assert int(err) == K.KV_DEV_ERR_PAGE_RANGE


def test_decode_mod_capped_scores_of_every_size():
    """Scores far above the cap, infinite products and a negative scale."""
    c = _cache([130], 1, 128, 16, "bf16", seed=8)
    q = (100 * torch.randn((1, 4, 128), generator=c["g"], device="cuda")).to(torch.bfloat16)
    for scale in (128**-0.5, -0.3, 30.0):
        ref, top = _reference(c, q, np.arange(1), np.array([129]), scale, 2.0)
        _close(_decode(c, q, scale, 1, softcap=2.0), ref, top, f"scale {scale}")


# ------------------------------------------------------------------ prefill
def _prefill(c, q, chunks, scale, key_start=None, prefix=None, max_q_len=None, err=None, out=None, **mod):
    start = np.concatenate([[0], np.cumsum(chunks)])
    out = torch.full(q.shape, float("nan"), device="cuda") if out is None else out
    K.paged_prefill_attention_mod(out, q, _d(start), int(max(chunks)) if max_q_len is None else max_q_len, c["kp"], c["vp"],
                                  torch.from_numpy(c["tab"]).cuda(), _d(c["lens"]), scale, err_flag=err,
                                  key_start=_d(key_start), prefix_lens=_d(prefix), **mod)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


PMODS = [dict(), dict(softcap=5.0), dict(window=40), dict(alibi=True), dict(docs=True), dict(prefix=True),
         dict(softcap=50.0, alibi=True, docs=True), dict(window=1), dict(window=150, prefix=True, alibi=True),
         dict(softcap=0.7, window=64, docs=True, prefix=True)]
PSHAPES = [("bf16", 128, 16, 32, 8, None), ("fp16", 128, 32, 16, 4, None), ("bf16", 128, 16, 8, 8, None),
           ("fp16", 128, 16, 64, 1, None), ("bf16", 64, 32, 16, 4, None), ("fp16", 64, 16, 12, 4, None),
           ("bf16", 128, 16, 28, 4, None), ("fp16", 128, 32, 32, 8, K.KV_DECODE_KERNEL_MMA)]


@pytest.mark.parametrize("mod", PMODS, ids=str)
@pytest.mark.parametrize("dtype,Dh,P,H_q,H_kv,kernel", PSHAPES)
def test_prefill_mod(dtype, Dh, P, H_q, H_kv, kernel, mod):
    lens, chunks = [400, 233, 95, 40, 1, 130], np.array([70, 64, 95, 17, 1, 3])
    c = _cache(lens, H_kv, Dh, P, dtype, seed=H_q + Dh)
    b, pos, _ = _rows(lens, chunks)
    q = (2 * torch.randn((len(b), H_q, Dh), generator=c["g"], device="cuda")).to(DT[dtype])
    rng = np.random.default_rng(1)
    ks = None
    if mod.get("docs"):
        ks = np.maximum(0, pos - rng.integers(0, 120, len(pos)))
        ks[::9] = -4
        ks[5::13] = pos[5::13] + 1 + rng.integers(0, 9)  # rows that see nothing (without a prefix)
        ks[200] = 10**9
    sl = _slopes(H_q) if mod.get("alibi") else None
    prefix = [0, 200, 1000, 30, 1, -5] if mod.get("prefix") else None
    cap, win = mod.get("softcap", 0.0), mod.get("window", 0)
    ref, top = _reference(c, q, b, pos, Dh**-0.5, cap, sl, win, ks, prefix)
    if kernel is not None:
        K.paged_decode_set_kernel(kernel)
    try:
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _prefill(c, q, chunks, Dh**-0.5, ks, prefix, err=err, softcap=cap, alibi_slopes=sl, window=win)
    finally:
        K.paged_decode_set_kernel(K.KV_DECODE_KERNEL_AUTO)
    assert int(err) == 0
    _close(got, ref, top, str(mod))


@pytest.mark.parametrize("kernel", [K.KV_DECODE_KERNEL_AUTO, K.KV_DECODE_KERNEL_MMA])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prefill_mod_hidden_values_and_visible_nan(dtype, kernel):
    """A NaN or infinity in V reaches the rows that see its key and no other row of the tile; in K likewise."""
    lens, chunks = [300, 180], np.array([90, 64])
    c = _cache(lens, 2, 128, 16, dtype, seed=12)
    b, pos, start = _rows(lens, chunks)
    q = torch.randn((len(b), 8, 128), generator=c["g"], device="cuda").to(DT[dtype])
    _put(c, 0, 250, 0, float("inf"), ("vp",))     # rows at 250 and behind see it
    _put(c, 0, 262, 1, float("nan"))
    page, off = int(c["tab"][1, 140 // 16]), 140 % 16
    c["vp"][page, 0, off, 7] = float("-inf")      # one element only
    _put(c, 1, 100, 1, float("nan"), ("vp",))     # behind the window of later rows
    ks = np.where(b == 0, 0, np.maximum(0, pos - 30))
    ref, top = _reference(c, q, b, pos, 128**-0.5, 20.0, None, 45, ks)
    assert np.isfinite(ref).any() and np.isnan(ref).any() and np.isinf(ref).any()
    K.paged_decode_set_kernel(kernel)
    try:
        got = _prefill(c, q, chunks, 128**-0.5, ks, softcap=20.0, window=45)
    finally:
        K.paged_decode_set_kernel(K.KV_DECODE_KERNEL_AUTO)
    _close(got, ref, top, "hidden values")


def test_prefill_mod_plain_options_equal_the_plain_entry_point():
    lens, chunks = [700, 95], np.array([100, 95])
    c = _cache(lens, 8, 128, 16, "bf16", seed=13)
    b, pos, start = _rows(lens, chunks)
    q = torch.randn((len(b), 32, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    got = _prefill(c, q, chunks, 128**-0.5)
    out = torch.empty(q.shape, device="cuda")
    K.paged_prefill_attention(out, q, _d(start), 100, c["kp"], c["vp"], torch.from_numpy(c["tab"]).cuda(), _d(lens), 128**-0.5)
    torch.cuda.synchronize()
    assert np.abs(got - out.double().cpu().numpy()).max() < 2.0**-13 * 5  # |v| < 5: the bound of _close on both sides


def test_prefill_mod_one_token_chunks_equal_decode():
    lens = [300, 47, 1000]
    c = _cache(lens, 8, 128, 16, "bf16", seed=14)
    q = torch.randn((3, 32, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    mod = dict(softcap=8.0, alibi_slopes=_slopes(32), window=64)
    a, d = _prefill(c, q, np.ones(3, int), 128**-0.5, **mod), _decode(c, q, 128**-0.5, 0, **mod)
    assert np.abs(a - d).max() < 2.0**-12 * 5


@pytest.mark.parametrize("Dh", [64, 128])
def test_prefill_mod_rows_left_alone_and_errors(Dh):
    lens, chunks = [20, 10, 33], np.array([5, 12, 8])  # the second chunk is longer than its sequence
    c = _cache(lens, 2, Dh, 16, "bf16", seed=15)
    q = torch.randn((40, 8, Dh), generator=c["g"], device="cuda").to(torch.bfloat16)
    out = torch.full(q.shape, 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _prefill(c, q, chunks, Dh**-0.5, out=out, err=err, window=6)
    assert int(err) == K.KV_DEV_ERR_SEQ_LEN
    assert (got[25:] == 7).all() and not got[5:17].any()
    b = np.repeat([0, 2], [5, 8])
    pos = np.r_[15:20, 25:33]
    rows = np.r_[0:5, 17:25]
    ref, top = _reference(c, q[torch.from_numpy(rows).cuda()], b, pos, Dh**-0.5, 0.0, None, 6)
    _close(got[rows], ref, top, "valid chunks")


def test_prefill_mod_long_context_and_repeats():
    lens, chunks = [6000, 2500], np.array([300, 1])
    c = _cache(lens, 2, 128, 16, "bf16", seed=16)
    b, pos, start = _rows(lens, chunks)
    q = torch.randn((len(b), 8, 128), generator=c["g"], device="cuda").to(torch.bfloat16)
    mod = dict(softcap=30.0, window=1000)
    first = _prefill(c, q, chunks, 128**-0.5, **mod)
    rows = np.r_[0, 1, 127, 128, 299, 300]
    ref, top = _reference(c, q[torch.from_numpy(rows).cuda()], b[rows], pos[rows], 128**-0.5, 30.0, None, 1000)
    _close(first[rows], ref, top, "long context")
    for _ in range(10):
        assert np.array_equal(_prefill(c, q, chunks, 128**-0.5, **mod), first)


def test_mod_layer_run():
    """A layer of capped, windowed attention as a server runs it: norm + rotation + append of a prompt chunk, chunked
    prefill, then decode steps replayed from one CUDA graph on a side stream."""
    from oracle.rope import rope_table

    H_q, H_kv, Dh, P, L = 16, 4, 128, 16, 75
    g = torch.Generator(device="cuda").manual_seed(20)
    pool = K.KvPool(20, P)
    tab = np.full((1, 8), -1, np.int32)
    tab[0, :-(-L // P)] = pool.alloc(-(-L // P))
    kp = torch.full((20, H_kv, P, Dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    cos_sin = torch.from_numpy(rope_table(256, Dh)).cuda()
    w = 1 + 0.1 * torch.randn(Dh, generator=g, device="cuda")
    mod = dict(softcap=30.0, window=32)

    def split(qkv):
        return qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]

    def c():
        return dict(lens=lens_h.copy(), tab=tab, kp=kp, vp=vp, P=P, H_kv=H_kv, Dh=Dh)

    qkv = torch.randn((L, H_q + 2 * H_kv, Dh), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = split(qkv)
    q_rot = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    K.kv_norm_rope_append(kp, vp, k, v, torch.from_numpy(K.kv_slots_for_range(tab[0], P, 0, L)).cuda(),
                          torch.arange(L, dtype=torch.int32, device="cuda"), cos_sin, w, 1e-6, P, q=q, q_out=q_rot, q_weight=w)
    lens_h = np.array([L], np.int32)
    got = _prefill(c(), q_rot, np.array([L]), Dh**-0.5, **mod)
    ref, top = _reference(c(), q_rot, np.zeros(L, int), np.arange(L), Dh**-0.5, 30.0, None, 32)
    _close(got, ref, top, "prompt")

    d_qkv = torch.empty((1, H_q + 2 * H_kv, Dh), dtype=torch.bfloat16, device="cuda")
    d_slot, d_pos, d_lens = (torch.zeros(1, dtype=t, device="cuda") for t in (torch.int64, torch.int32, torch.int32))
    d_tab = torch.from_numpy(tab).cuda()
    d_q = torch.empty((1, H_q, Dh), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((1, H_q, Dh), device="cuda")
    ws = torch.empty(max(16, K.paged_decode_ext_workspace_bytes(1, H_q, H_kv, Dh, 8, P)), dtype=torch.uint8, device="cuda")
    d_slot.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        dq, dk, dv = split(d_qkv)
        K.kv_norm_rope_append(kp, vp, dk, dv, d_slot, d_pos, cos_sin, w, 1e-6, P, q=dq, q_out=d_q, q_weight=w)
        K.paged_decode_attention_mod(out, d_q, kp, vp, d_tab, d_lens, Dh**-0.5, workspace=ws, **mod)
    for step in range(8):
        d_slot.copy_(torch.from_numpy(pool.append_slots(tab, lens_h)))
        d_tab.copy_(torch.from_numpy(tab))
        d_lens.copy_(torch.from_numpy(lens_h))
        d_pos.copy_(d_lens - 1)
        d_qkv.copy_(torch.randn(d_qkv.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ref, top = _reference(c(), d_q, np.zeros(1, int), lens_h - 1, Dh**-0.5, 30.0, None, 32)
        _close(out.double().cpu().numpy(), ref, top, f"step {step}")
