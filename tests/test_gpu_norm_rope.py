"""GPU parity of kv_norm_rope_append (per-head RMS norm, rotation, append in one pass) against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import score_mod as O
from oracle.rope import rope_table
from paged_kv_cache_433_b200 import kvpaged as K

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_433_b200 import build

    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _close(got, ref, dtype, what):
    """One rounding to the storage type (half a step, eps / 2 of the value; below the type's normal range half the
    subnormal step) on top of fp32 arithmetic: the sum of Dh squares, its root and quotient, two products and the
    rotation's three operations err by at most (Dh + 16) * 2^-24 of the row's largest element."""
    info = torch.finfo(DT[dtype])
    top = np.abs(ref).max(-1, keepdims=True)
    tol = np.abs(ref) * info.eps / 2 + info.tiny * info.eps / 2 + (ref.shape[-1] + 16) * 2.0**-24 * top
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: {(err > tol).sum()} outside, worst {np.max(err / tol):.2f} of the bound"


def _case(B, H_q, H_kv, Dh, P, dtype, style, fused, seed=0, bad=False, weights=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    max_pos = 500
    if fused:
        qkv = rnd(B, H_q + 2 * H_kv, Dh)
        q, k, v = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
    else:
        q, k, v = rnd(B, H_q, Dh), rnd(B, H_kv, Dh), rnd(B, H_kv, Dh)
    num_pages = -(-B // P) + 3
    slots = torch.randperm(num_pages * P, generator=g, device="cuda")[:B].contiguous()
    pos = torch.randint(0, max_pos, (B,), generator=g, device="cuda").to(torch.int32)
    if bad:
        slots[0], slots[1], pos[2], pos[3] = -1, num_pages * P, -1, max_pos
    tab = torch.from_numpy(rope_table(max_pos, Dh)).cuda()
    wq = 1 + 0.2 * torch.randn(Dh, generator=g, device="cuda") if weights else None
    wk = 1 + 0.2 * torch.randn(Dh, generator=g, device="cuda") if weights else None
    kp, vp = rnd(num_pages, H_kv, P, Dh), rnd(num_pages, H_kv, P, Dh)
    return dict(q=q, k=k, v=v, slots=slots, pos=pos, tab=tab, wq=wq, wk=wk, kp=kp, vp=vp, P=P, style=style, dtype=dtype,
                max_pos=max_pos, num_pages=num_pages)


def _reference(c, eps):
    n = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    pos = c["pos"].cpu().numpy()
    safe = np.clip(pos, 0, c["max_pos"] - 1)
    q = O.norm_rope(n(c["q"]), n(c["wq"]), eps, safe, n(c["tab"]), c["style"])
    k = O.norm_rope(n(c["k"]), n(c["wk"]), eps, safe, n(c["tab"]), c["style"])
    return q, k, (pos >= 0) & (pos < c["max_pos"])


def _check(c, eps=1e-6, err_bits=0):
    P = c["P"]
    q_ref, k_ref, pos_ok = _reference(c, eps)
    kp0, vp0 = c["kp"].clone(), c["vp"].clone()
    q_out = torch.full(c["q"].shape, 7.0, dtype=DT[c["dtype"]], device="cuda")
    k_out = torch.full(c["k"].shape, 7.0, dtype=DT[c["dtype"]], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kv_norm_rope_append(c["kp"], c["vp"], c["k"], c["v"], c["slots"], c["pos"], c["tab"], c["wk"], eps, P, style=c["style"],
                          q=c["q"], q_out=q_out, q_weight=c["wq"], k_out=k_out, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == err_bits
    d = c["dtype"]
    _close(q_out.double().cpu().numpy()[pos_ok], q_ref[pos_ok], d, "q")
    _close(k_out.double().cpu().numpy()[pos_ok], k_ref[pos_ok], d, "k_out")
    assert (q_out[torch.from_numpy(~pos_ok).cuda()] == 7).all() and (k_out[torch.from_numpy(~pos_ok).cuda()] == 7).all()
    slots = c["slots"].cpu().numpy()
    wrote = pos_ok & (slots >= 0) & (slots < c["num_pages"] * P)
    sl, rows = torch.from_numpy(slots[wrote]).cuda(), torch.from_numpy(np.nonzero(wrote)[0]).cuda()
    kp0[sl // P, :, sl % P] = k_out[rows]  # the page rows hold the bits of k_out; every other row its old bits
    vp0[sl // P, :, sl % P] = c["v"][rows]
    assert torch.equal(c["kp"], kp0) and torch.equal(c["vp"], vp0)


SHAPES = [  # B, H_q, H_kv, Dh, P, dtype, style, fused
    (1, 32, 8, 128, 16, "bf16", "half", True), (64, 32, 8, 128, 16, "bf16", "half", True),
    (777, 32, 8, 128, 32, "fp16", "interleaved", True), (5, 6, 2, 64, 16, "fp16", "half", False),
    (333, 7, 7, 64, 32, "bf16", "interleaved", True), (40, 4, 1, 256, 16, "fp32", "half", True),
    (3, 64, 8, 512, 16, "bf16", "half", True), (9, 3, 1, 16, 16, "bf16", "interleaved", True),
    (2000, 128, 16, 128, 16, "bf16", "half", True),  # more row pieces than threads, more tokens than CTAs
    (65, 2, 2, 128, 16, "fp32", "interleaved", False),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_norm_rope_append(shape):
    _check(_case(*shape))


def test_norm_rope_without_weights_and_bad_tokens():
    _check(_case(70, 8, 2, 128, 16, "bf16", "half", True, bad=True, weights=False),
           err_bits=K.KV_DEV_ERR_SLOT | K.KV_DEV_ERR_POSITION)


def test_norm_rope_small_rows_take_eps():
    c = _case(20, 8, 2, 128, 16, "fp32", "half", False)
    c["q"] *= 1e-5
    c["k"].zero_()
    _check(c, eps=1e-5)


def test_norm_rope_k_only_and_in_place():
    c = _case(50, 8, 2, 128, 16, "bf16", "half", False)
    q_ref, k_ref, _ = _reference(c, 1e-6)
    K.kv_norm_rope_append(None, None, c["k"], None, None, c["pos"], c["tab"], c["wk"], 1e-6, 16, q=c["q"], q_out=c["q"],
                          q_weight=c["wq"], k_out=c["k"])
    torch.cuda.synchronize()
    _close(c["q"].double().cpu().numpy(), q_ref, "bf16", "q in place")
    _close(c["k"].double().cpu().numpy(), k_ref, "bf16", "k in place")


def test_norm_rope_refuses_in_place_slices_and_other_layouts():
    c = _case(4, 8, 2, 128, 16, "bf16", "half", True)
    call = lambda **kw: K.kv_norm_rope_append(**{**dict(  # noqa: E731
        k_pages=c["kp"], v_pages=c["vp"], k_new=c["k"], v_new=c["v"], slot_mapping=c["slots"], positions=c["pos"],
        cos_sin=c["tab"], k_weight=c["wk"], eps=1e-6, page_size=16), **kw})
    with pytest.raises(ValueError):
        call(q=c["q"], q_out=c["q"])  # a slice cannot be the contiguous output
    with pytest.raises(ValueError):
        call(k_new=c["k"].transpose(1, 2).contiguous().transpose(1, 2))  # heads not contiguous
    with pytest.raises(ValueError):
        call(k_new=c["k"].float())
    with pytest.raises(ValueError):
        call(positions=c["pos"][:2])
    with pytest.raises(K.KvError):
        call(k_new=c["k"][:1].expand(4, 2, 128))  # stride 0


def test_norm_rope_graph_and_side_stream():
    c = _case(64, 32, 8, 128, 16, "bf16", "half", True)
    q_ref, k_ref, _ = _reference(c, 1e-6)
    q_out = torch.zeros(c["q"].shape, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        K.kv_norm_rope_append(c["kp"], c["vp"], c["k"], c["v"], c["slots"], c["pos"], c["tab"], c["wk"], 1e-6, 16,
                              q=c["q"], q_out=q_out, q_weight=c["wq"])
    for _ in range(2):
        q_out.zero_()
        g.replay()
        torch.cuda.synchronize()
        _close(q_out.double().cpu().numpy(), q_ref, "bf16", "q replayed")
