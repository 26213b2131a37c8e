"""GPU parity of the int8 K/V cache: quantising append (bit-exact codes and scales), page read-back, page copy, decode
attention, against the oracle."""
import numpy as np
import pytest
import torch

from oracle import score_mod as O
from paged_kv_cache_433_b200 import kvpaged as K

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_433_b200 import build

    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pools(num_pages, H_kv, P, Dh, g):
    codes = torch.randint(-127, 128, (2, num_pages, H_kv, P, Dh), generator=g, device="cuda", dtype=torch.int16)
    scales = torch.rand((num_pages, H_kv, 2, P), generator=g, device="cuda") + 0.01
    return codes[0].to(torch.int8), codes[1].to(torch.int8), scales


@pytest.mark.parametrize("B,H_kv,Dh,P,dtype,strided", [
    (1, 8, 128, 16, "bf16", False), (64, 8, 128, 16, "bf16", True), (1000, 2, 64, 32, "fp16", True), (7, 3, 16, 16, "fp32", False),
    (33, 1, 512, 16, "bf16", True), (3001, 8, 128, 32, "fp32", True)])
def test_append_bits(B, H_kv, Dh, P, dtype, strided):
    g = _gen(B)
    num_pages = -(-B // P) + 2
    kp, vp, sc = _pools(num_pages, H_kv, P, Dh, g)
    x = (torch.randn((B, 2 * H_kv, Dh), generator=g, device="cuda") * torch.exp(
        4 * torch.randn((B, 2 * H_kv, 1), generator=g, device="cuda"))).to(DT[dtype])
    if B > 5:  # rows that are zero, too small for a scale, or not finite
        x[0, 0] = 0
        x[1, 1] = 2.0**-126 if dtype != "fp16" else 0
        x[2, 0, Dh // 2] = float("nan")
        x[3, 2 * H_kv - 1, 3] = float("-inf")
        x[4] = torch.round(x[4].float().clamp(-100, 100) * 2).to(DT[dtype]) / 2  # ties
        x[4, :, 0] = 127
    k, v = x[:, :H_kv], x[:, H_kv:]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    slots = torch.randperm(num_pages * P, generator=g, device="cuda")[:B].contiguous()
    err_want = 0
    if B > 9:
        slots[7], slots[8], err_want = -1, num_pages * P + 5, K.KV_DEV_ERR_SLOT
    want = [t.cpu().numpy().copy() for t in (kp, vp, sc)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kv_append_int8(kp, vp, sc, k, v, slots, P, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == err_want
    sl = slots.cpu().numpy()
    ok = (sl >= 0) & (sl < num_pages * P)
    for i, (t, pages) in enumerate(((k, want[0]), (v, want[1]))):
        codes, scales = O.quantise_int8(t.float().cpu().numpy())
        pages[sl[ok] // P, :, sl[ok] % P] = codes[ok]
        want[2][sl[ok] // P, :, i, sl[ok] % P] = scales[ok]
    assert np.array_equal(kp.cpu().numpy(), want[0]) and np.array_equal(vp.cpu().numpy(), want[1])
    assert np.array_equal(sc.cpu().numpy(), want[2], equal_nan=True)


@pytest.mark.parametrize("H_kv,Dh,P,dtype,n", [(8, 128, 16, "bf16", 9), (3, 64, 32, "fp16", 1), (2, 128, 16, "fp32", 40),
                                               (1, 80, 5, "bf16", 3), (16, 512, 32, "bf16", 2)])
def test_dequant_and_copy_pages(H_kv, Dh, P, dtype, n):
    g = _gen(n)
    num_pages, num_out = 2 * n + 5, n + 4
    kp, vp, sc = _pools(num_pages, H_kv, P, Dh, g)
    src = torch.randint(0, num_pages, (n,), generator=g, device="cuda").to(torch.int32)  # a page may be read twice
    dst = torch.randperm(num_out, generator=g, device="cuda")[:n].to(torch.int32)
    ko = torch.full((num_out, H_kv, P, Dh), 3.0, dtype=DT[dtype], device="cuda")
    vo = ko.clone()
    bad = 0
    s_l, d_l = src.long(), dst.long()
    if n > 8:
        src[0], src[1], dst[2], bad = -1, num_pages, num_out, K.KV_DEV_ERR_PAGE_RANGE
        s_l, d_l = s_l[3:], d_l[3:]
    want_k, want_v = ko.clone(), vo.clone()
    want_k[d_l] = (kp[s_l].float() * sc[s_l, :, 0][..., None]).to(DT[dtype])
    want_v[d_l] = (vp[s_l].float() * sc[s_l, :, 1][..., None]).to(DT[dtype])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kv_dequant_pages_int8(ko, vo, kp, vp, sc, src, dst, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == bad and torch.equal(ko, want_k) and torch.equal(vo, want_v)

    if (H_kv * P) % 2 == 0:
        perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
        cs, cd = perm[:n].contiguous(), perm[n:2 * n].contiguous()
        want = [t.clone() for t in (kp, vp, sc)]
        for t in want:
            t[cd.long()] = t[cs.long()]
        K.kv_copy_pages_int8(kp, vp, sc, cs, cd, err_flag=err.zero_())
        torch.cuda.synchronize()
        assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip((kp, vp, sc), want))
        K.kv_copy_pages_int8(kp, vp, sc, torch.tensor([-1], dtype=torch.int32, device="cuda"), cd[:1], err_flag=err)
        torch.cuda.synchronize()
        assert int(err) == K.KV_DEV_ERR_PAGE_RANGE and all(torch.equal(a, b) for a, b in zip((kp, vp, sc), want))


def _decode_case(lens, H_q, H_kv, Dh, P, dtype, seed=0, q_scale=1.0, poison=True):
    """A cache of random pages; unused slots hold NaN scales, unused table entries -1."""
    g = _gen(seed)
    lens = np.asarray(lens)
    need = -(-lens // P)
    mb = max(1, int(need.max()))
    num_pages = int(need.sum()) + 2
    kp, vp, sc = _pools(num_pages, H_kv, P, Dh, g)
    sc = (sc * torch.exp(torch.randn(sc.shape, generator=g, device="cuda"))) / 127
    order = torch.randperm(num_pages, generator=g, device="cuda").cpu().numpy()
    tab = np.full((len(lens), mb), -1, np.int32)
    used = np.zeros((num_pages, P), bool)
    at = 0
    for b, L in enumerate(lens):
        tab[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = np.arange(L)
        used[tab[b][t // P], t % P] = True
    if poison:
        sc.masked_fill_(torch.from_numpy(~used).cuda()[:, None, None, :], float("nan"))
    q = (torch.randn((len(lens), H_q, Dh), generator=g, device="cuda") * q_scale).to(DT[dtype])
    return dict(lens=lens, tab=tab, kp=kp, vp=vp, sc=sc, q=q, P=P, H_q=H_q, H_kv=H_kv, Dh=Dh, scale=Dh**-0.5 / q_scale)


def _reference(c, rows=None):
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    kp, vp, sc, q = n(c["kp"]), n(c["vp"]), n(c["sc"]), n(c["q"])
    k_all, v_all = kp * sc[:, :, 0][..., None], vp * sc[:, :, 1][..., None]
    out = np.zeros(q.shape)
    top = np.zeros((len(q), 1, 1))
    for b, L in enumerate(c["lens"]):
        if rows is not None and b not in rows:
            continue
        k, v = (O.gather(x, c["tab"][b], int(L), c["P"]) for x in (k_all, v_all))
        if L:
            out[b] = O.attend_row(q[b], k, v, int(L) - 1, int(L), c["scale"])
            top[b] = np.abs(v).max()
    return out, top


def _decode(c, num_splits=0, err=None, out=None):
    B = len(c["lens"])
    out = torch.full((B, c["H_q"], c["Dh"]), float("nan"), device="cuda") if out is None else out
    need = K.paged_decode_ext_workspace_bytes(B, c["H_q"], c["H_kv"], c["Dh"], c["tab"].shape[1], c["P"], num_splits)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    K.paged_decode_attention_int8(out, c["q"], c["kp"], c["vp"], c["sc"], torch.from_numpy(c["tab"]).cuda(),
                                  torch.from_numpy(c["lens"].astype(np.int32)).cuda(), c["scale"], num_splits=num_splits,
                                  workspace=ws, err_flag=err)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def _close(got, ref, top, what, rows=slice(None)):
    """Weights go into the product as a bf16 value and its rounded residual (2^-17 of each weight at most), scores err
    by a few 2^-22 of their size (below 30 in these cases), sums by 2^-23 a step of 16 keys: 2^-14 of the largest
    visible |v| bounds their sum."""
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref)
    assert (err <= 2.0**-14 * top)[rows].all(), f"{what}: worst {np.max(err / np.maximum(top, 1e-30)):.2e} of max |v|"


SHAPES = [("bf16", 128, 16, 32, 8), ("fp16", 128, 16, 32, 8), ("bf16", 128, 32, 8, 8), ("fp16", 64, 16, 6, 2),
          ("bf16", 64, 32, 16, 1), ("bf16", 128, 16, 64, 1), ("fp16", 128, 32, 28, 4)]


@pytest.mark.parametrize("num_splits", [1, 0, 3])
@pytest.mark.parametrize("dtype,Dh,P,H_q,H_kv", SHAPES)
def test_decode_int8(dtype, Dh, P, H_q, H_kv, num_splits):
    c = _decode_case([1, 0, P, P + 1, 2 * P - 1, 300, 517, 1029], H_q, H_kv, Dh, P, dtype, seed=H_q)
    ref, top = _reference(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _close(_decode(c, num_splits, err), ref, top, f"S={num_splits}")
    assert int(err) == 0


def test_decode_int8_planned_many_rows():
    g = np.random.default_rng(5)
    lens = np.rint(np.exp(g.normal(4.5, 1.0, 160))).astype(int).clip(0, 900)
    lens[3] = 0
    c = _decode_case(lens, 32, 8, 128, 16, "bf16", seed=9)
    rows = list(range(0, 160, 7)) + [3]
    ref, top = _reference(c, rows)
    _close(_decode(c), ref, top, "planned", rows)


@pytest.mark.parametrize("q_scale", [1e-30, 1e-4, 1e4, 1e30])
def test_decode_int8_takes_any_bf16_query(q_scale):
    c = _decode_case([200, 33], 8, 2, 128, 16, "bf16", seed=2, q_scale=q_scale)
    ref, top = _reference(c)
    _close(_decode(c, 1), ref, top, "q scale")


def test_decode_int8_wide_scales():
    """Scales from 2^-60 to 2^60 across tokens: the weighted codes keep their precision in the product."""
    c = _decode_case([400, 37], 8, 2, 128, 16, "fp16", seed=4, poison=False)
    e = torch.randint(-60, 61, c["sc"][:, :, 1].shape, generator=_gen(1), device="cuda").float()
    c["sc"][:, :, 1] = torch.exp2(e)
    ref, top = _reference(c)
    _close(_decode(c, 1), ref, top, "wide scales")


def test_decode_int8_bad_pages_and_lengths():
    """A bad table entry skips its own page only (pages of 16 share a stage in pairs); a bad length gives zeros."""
    c = _decode_case([100, 64, 50], 8, 2, 128, 16, "bf16", seed=6)
    c["tab"][0, 2] = 10**6
    c["tab"][1, 1] = -5
    keep = {0: np.r_[0:32, 48:100], 1: np.r_[0:16, 32:64]}
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    kp, vp, sc, q = n(c["kp"]), n(c["vp"]), n(c["sc"]), n(c["q"])
    safe = np.clip(c["tab"], 0, len(kp) - 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["lens"] = np.array([100, 64, 10**6])
    got = _decode(c, 1, err)
    assert int(err) == K.KV_DEV_ERR_PAGE_RANGE | K.KV_DEV_ERR_SEQ_LEN
    assert not got[2].any()
    for b, t in keep.items():
        k = (kp * sc[:, :, 0][..., None])[safe[b][t // 16], :, t % 16]
        v = (vp * sc[:, :, 1][..., None])[safe[b][t // 16], :, t % 16]
        ref = O.attend_row(q[b], k, v, len(t) - 1, len(t), c["scale"])
        _close(got[b], ref, np.abs(v).max(), f"row {b}")


@pytest.mark.parametrize("num_splits", [1, 4])
def test_decode_int8_nan_scale_shows(num_splits):
    c = _decode_case([100, 90], 8, 2, 128, 16, "bf16", seed=7)
    c["sc"][int(c["tab"][0, 1]), 1, 0, 3] = float("nan")  # K of head 1, token 19 of row 0
    c["sc"][int(c["tab"][1, 2]), 0, 1, 5] = float("nan")  # V of head 0, token 37 of row 1
    got = _decode(c, num_splits)
    assert np.isnan(got[0, 4:]).all() and np.isfinite(got[0, :4]).all()
    assert np.isnan(got[1, :4]).all() and np.isfinite(got[1, 4:]).all()


def test_decode_int8_repeats_and_graph():
    c = _decode_case([700, 3, 0, 250], 32, 8, 128, 16, "bf16", seed=8)
    tab, lens = torch.from_numpy(c["tab"]).cuda(), torch.from_numpy(c["lens"].astype(np.int32)).cuda()
    out = torch.empty((4, 32, 128), device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    call = lambda: K.paged_decode_attention_int8(out, c["q"], c["kp"], c["vp"], c["sc"], tab, lens, c["scale"],  # noqa: E731
                                                 num_splits=3, workspace=ws)
    call()
    torch.cuda.synchronize()
    first = out.clone()
    ref, top = _reference(c)
    _close(first.double().cpu().numpy(), ref, top, "first")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(20):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_int8_serving_run():
    """A prompt written to the int8 cache and read back for the 16-bit chunked prefill of its tail, then decode steps
    over the int8 pages with the norm + rotation in front, as a server would run them."""
    from oracle.rope import rope_table

    g = _gen(11)
    H_q, H_kv, Dh, P, L, n_new = 16, 4, 128, 16, 150, 3
    pool = K.KvPool(24, P)
    tab = np.full((1, 16), -1, np.int32)
    tab[0, :-(-L // P)] = pool.alloc(-(-L // P))
    kp = torch.zeros((24, H_kv, P, Dh), dtype=torch.int8, device="cuda")
    vp, sc = torch.zeros_like(kp), torch.zeros((24, H_kv, 2, P), device="cuda")
    cos_sin = torch.from_numpy(rope_table(512, Dh)).cuda()
    wq, wk = (1 + 0.1 * torch.randn(Dh, generator=g, device="cuda") for _ in range(2))
    n = lambda t: t.double().cpu().numpy()  # noqa: E731

    def write(qkv, pos, slots):
        q, k, v = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
        q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        k_rot = torch.empty(k.shape, dtype=k.dtype, device="cuda")
        K.kv_norm_rope_append(None, None, k, None, None, pos, cos_sin, wk, 1e-6, P, q=q, q_out=q_out, q_weight=wq, k_out=k_rot)
        K.kv_append_int8(kp, vp, sc, k_rot, v, slots, P)
        return q_out

    qkv = torch.randn((L, H_q + 2 * H_kv, Dh), generator=g, device="cuda").to(torch.bfloat16)
    q = write(qkv, torch.arange(L, device="cuda", dtype=torch.int32),
              torch.from_numpy(K.kv_slots_for_range(tab[0], P, 0, L)).cuda())
    # read back into a 16-bit scratch pool and run the last 40 tokens as a chunk
    nb = -(-L // P)
    k16 = torch.empty((nb, H_kv, P, Dh), dtype=torch.bfloat16, device="cuda")
    v16 = torch.empty_like(k16)
    ids = torch.arange(nb, dtype=torch.int32, device="cuda")
    K.kv_dequant_pages_int8(k16, v16, kp, vp, sc, torch.from_numpy(tab[0, :nb]).cuda(), ids)
    out = torch.empty((40, H_q, Dh), device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    K.paged_prefill_attention(out, q[-40:].contiguous(), torch.tensor([0, 40], dtype=torch.int32, device="cuda"), 40, k16, v16,
                              ids[None].contiguous(), lens, Dh**-0.5)
    torch.cuda.synchronize()
    k_log, v_log = (n(x).transpose(0, 2, 1, 3).reshape(-1, H_kv, Dh)[:L] for x in (k16, v16))
    ref = np.stack([O.attend_row(n(q[L - 40 + i]), k_log, v_log, L - 40 + i, L, Dh**-0.5) for i in range(40)])
    _close(out.double().cpu().numpy(), ref, np.abs(v_log).max() * 2, "prefill over read-back pages")
    lens_h = np.array([L], np.int32)
    for step in range(n_new):
        slots = pool.append_slots(tab, lens_h)
        qkv = torch.randn((1, H_q + 2 * H_kv, Dh), generator=g, device="cuda").to(torch.bfloat16)
        q = write(qkv, torch.tensor([int(lens_h[0]) - 1], dtype=torch.int32, device="cuda"), torch.from_numpy(slots).cuda())
        c = dict(lens=lens_h.copy(), tab=tab, kp=kp, vp=vp, sc=sc, q=q, P=P, H_q=H_q, H_kv=H_kv, Dh=Dh, scale=Dh**-0.5)
        ref, top = _reference(c)
        _close(_decode(c), ref, top, f"step {step}")
