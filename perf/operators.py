"""Workloads of the cache-side and score-side operators next to paged attention.

Five operators, each as a serving step calls it: the per-head norm + rotation +
append of a step's q / k / v, writing an int8 cache and reading it back, decode
over that int8 cache, and decode and chunked prefill with modified scores and
masks (tanh cap, distance bias, sliding window, documents, bidirectional
prefix). `run` computes them in elementary torch operations in 32 bits, or,
where `own` is true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
# the scratch a serving program keeps for split partials, one for all its calls
WORKSPACE_BYTES = 64 << 20


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 sequences, 8B-shaped layer: q/k/v are slices of the fused projection's output
        dict(name="norm_rope-step-B64-bf16", op="norm_rope", T=64, H_q=32, H_kv=8, Dh=128, P=16, dtype="bf16", style="half"),
        # a prefill batch's 8192 prompt tokens, interleaved rotation
        dict(name="norm_rope-prompt-T8192-fp16", op="norm_rope", T=8192, H_q=32, H_kv=8, Dh=128, P=16, dtype="fp16",
             style="interleaved"),
        # one decode step written to the int8 cache, 64 tail pages read back
        dict(name="int8_cache-step-B64-bf16", op="int8_cache", T=64, pages=64, H_kv=8, Dh=128, P=16, dtype="bf16"),
        # a prompt written to the int8 cache, all its pages widened for a 16-bit prefill
        dict(name="int8_cache-prompt-T8185-bf16", op="int8_cache", T=8185, pages=512, H_kv=8, Dh=128, P=16, dtype="bf16"),
        # the 8B-shaped decode batch over int8 pages
        dict(name="decode_int8-B64-len512..4096-bf16", op="decode_int8", B=64, lo=512, hi=4096, H_q=32, H_kv=8, Dh=128, P=16,
             dtype="bf16"),
        # one long sequence over int8 pages
        dict(name="decode_int8-B1-T32768-fp16", op="decode_int8", B=1, lo=32768, hi=32768, H_q=32, H_kv=8, Dh=128, P=16,
             dtype="fp16"),
        # a single request in a sliding-window layer with capped scores (latency)
        dict(name="decode_mod-B1-len2000-window512-cap", op="decode_mod", B=1, lo=2000, hi=2000, H_q=32, H_kv=8, Dh=128, P=16,
             dtype="bf16", cap=50.0, window=512, alibi=False, docs=0),
        # the 8B-shaped decode batch in a global layer with capped scores
        dict(name="decode_mod-B64-len512..4096-cap", op="decode_mod", B=64, lo=512, hi=4096, H_q=32, H_kv=8, Dh=128, P=16,
             dtype="bf16", cap=50.0, window=0, alibi=False, docs=0),
        # many short and a few long sequences, distance bias and packed documents, many rows
        dict(name="decode_mod-B256-len16..8192-alibi-docs", op="decode_mod", B=256, lo=16, hi=8192, H_q=32, H_kv=8, Dh=128,
             P=32, dtype="fp16", cap=0.0, window=0, alibi=True, docs=1024),
        # chunked prefill of a global layer with capped scores
        dict(name="prefill_mod-B8-ctx4096-chunk512-cap", op="prefill_mod", B=8, ctx_lo=4096, ctx_hi=4096, n_lo=512, n_hi=512,
             H_q=32, H_kv=8, Dh=128, P=16, dtype="bf16", cap=50.0, window=0, alibi=False, docs=0, prefix=0),
        # short ragged chunks (drafted tokens, prompt tails) with distance bias and a bidirectional prefix
        dict(name="prefill_mod-B6-ragged1..70-alibi-prefix", op="prefill_mod", B=6, ctx_lo=0, ctx_hi=700, n_lo=1, n_hi=70,
             H_q=16, H_kv=4, Dh=64, P=32, dtype="fp16", cap=0.0, window=0, alibi=True, docs=0, prefix=96),
        # whole prompts of packed documents in a sliding-window layer
        dict(name="prefill_mod-B2-n4096-docs-window1024", op="prefill_mod", B=2, ctx_lo=0, ctx_hi=0, n_lo=4000, n_hi=4096,
             H_q=32, H_kv=8, Dh=128, P=16, dtype="bf16", cap=30.0, window=1024, alibi=False, docs=1500, prefix=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "int8_cache", "decode_int8", "decode_mod", "decode_mod", "prefill_mod", "prefill_mod"])
    H_kv, g = rng.choice([(8, 4), (8, 4), (4, 8), (8, 1), (2, 3), (1, 16), (4, 7), (8, 8)])
    c = dict(op=op, H_q=H_kv * g, H_kv=H_kv, Dh=rng.choice([64, 128, 128]), P=rng.choice([16, 32]),
             dtype=rng.choice(["bf16", "fp16"]))
    if op == "norm_rope":
        c |= dict(T=_log(rng, 1, 6000), style=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "fp16", "fp32"]))
        c["T"] = max(1, min(c["T"], 8192 * 48 // (c["H_q"] + 2 * H_kv) // (2 if c["dtype"] == "fp32" else 1)))
    elif op == "int8_cache":
        c |= dict(T=_log(rng, 1, 8000))
        c["pages"] = -(-c["T"] // c["P"])
        del c["H_q"]
    elif op == "decode_int8":
        B = _log(rng, 1, 96)
        hi = _log(rng, 1, max(1, min(32768, 140000 // B)))
        c |= dict(B=B, lo=max(1, hi // rng.choice([1, 4, 100])), hi=hi)
    else:
        c |= dict(cap=rng.choice([0.0, 20.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, 3000)]), alibi=rng.random() < 0.4,
                  docs=rng.choice([0, 0, _log(rng, 8, 2000)]))
        if op == "decode_mod":
            B = _log(rng, 1, 300)
            hi = _log(rng, 1, max(1, min(32768, 260000 // B)))
            c |= dict(B=B, lo=max(1, hi // rng.choice([1, 4, 100])), hi=hi)
        else:
            B = _log(rng, 1, 12)
            n = _log(rng, 1, 3000 // B)
            ctx = _log(rng, 1, 4000)
            c |= dict(B=B, n_lo=max(1, n // rng.choice([1, 3, 50])), n_hi=n, ctx_lo=ctx // rng.choice([1, 4]), ctx_hi=ctx,
                      prefix=rng.choice([0, 0, _log(rng, 1, 2000)]))
    return c


def _ints(case, what, n, lo, hi):
    """n lengths between lo and hi (log-uniform), the same for a case whatever its values are."""
    r = np.random.RandomState((_hash(case) + what) % (1 << 32))
    return np.rint(np.exp(r.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)), n))).astype(np.int64).clip(lo, hi)


def _hash(case):
    h = 2166136261
    for k in sorted(case):
        if k != "name":
            for ch in ("%s=%s;" % (k, case[k])).encode():
                h = (h ^ ch) * 16777619 % (1 << 32)
    return h


def _lens(case):
    """(total tokens, chunk tokens) of each sequence."""
    if case["op"] == "prefill_mod":
        n = _ints(case, 2, case["B"], case["n_lo"], case["n_hi"])
        return _ints(case, 1, case["B"], case["ctx_lo"], case["ctx_hi"]) + n, n
    lens = _ints(case, 1, case["B"], case["lo"], case["hi"])
    return lens, np.ones_like(lens)


def _rows(case):
    """For every query row, in order: its sequence, its position, and the interval [lo, hi) of keys that it sees
    (host arrays), with the first visible key that a document gives it."""
    total, n = _lens(case)
    b = np.repeat(np.arange(len(n)), n)
    start = np.concatenate([[0], np.cumsum(n)])
    pos = (total - n)[b] + np.arange(len(b)) - start[b]
    doc = np.zeros(len(b), np.int64)
    if case["docs"]:  # documents of `docs` tokens, cut anew in every sequence
        off = _ints(case, 3, len(n), 1, case["docs"])[b]
        doc = np.maximum(0, (pos + off) // case["docs"] * case["docs"] - off)
    lo = np.maximum(doc, pos - case["window"] + 1 if case["window"] else 0)
    hi = pos + 1
    if case.get("prefix"):
        hi = np.maximum(hi, np.minimum(_prefix(case), total)[b])
    return b, pos, lo, hi, doc, start


def _prefix(case):
    return _ints(case, 4, case["B"], 1, case["prefix"])


def work(case):
    op, H, D = case["op"], case["H_kv"], case["Dh"]
    if op == "norm_rope":
        T, e = case["T"], BYTES[case["dtype"]]
        rows = case["H_q"] + 2 * H
        return {"bytes": T * (2 * rows * D * e + 4 * D + 12) + 8 * D, "flops": T * (case["H_q"] + H) * D * 7}
    if op == "int8_cache":
        e, T, n = BYTES[case["dtype"]], case["T"], case["pages"] * case["P"]
        return {"bytes": 2 * T * H * (D * (e + 1) + 4) + 8 * T + 2 * n * H * (D * (1 + e) + 4),
                "flops": 2 * (3 * T + n) * H * D}
    Hq, e = case["H_q"], BYTES[case["dtype"]]
    if op == "decode_int8":
        keys = int(_lens(case)[0].sum())
        return {"bytes": keys * H * (2 * D + 8) + case["B"] * Hq * D * (e + 4), "flops": 4 * keys * Hq * D}
    b, pos, lo, hi, doc, start = _rows(case)
    seen = np.maximum(hi - lo, 0)
    pairs = int(seen.sum())
    first = np.full(case["B"], 1 << 60)
    last = np.zeros(case["B"], np.int64)
    np.minimum.at(first, b, lo)
    np.maximum.at(last, b, hi)
    keys = int(np.maximum(last - first, 0).sum())  # keys that some row of the sequence sees
    return {"bytes": 2 * keys * H * D * e + len(b) * Hq * D * (e + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DT[dtype])


def _table(case, g, lens):
    """A block table whose pages lie anywhere in the pool; entries behind a sequence's last page stay unused (-1)."""
    P = case["P"]
    need = -(-lens // P)
    mb = int(need.max())
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    used = torch.arange(mb)[None, :] < torch.from_numpy(need)[:, None]
    idx = torch.cumsum(used.reshape(-1), 0).reshape(used.shape) - 1
    tab = torch.where(used.cuda(), order[idx.cuda().clamp(min=0)], torch.tensor(-1, dtype=torch.int32, device="cuda"))
    return tab.contiguous(), pages


def _slots(case, g, T, extra):
    """Slots of T consecutive tokens over randomly ordered pages, those pages, and the pool's page count."""
    P = case["P"]
    n = -(-T // P)
    pages = n + extra
    order = torch.randperm(pages, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    return (order[t // P] * P + t % P).contiguous(), order[:n].to(torch.int32).contiguous(), pages


def _cos_sin(max_pos, Dh):
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
        torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -2.0 * torch.arange(Dh // 2, device="cuda") / Dh)[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, H, D, P, dt = case["op"], case["H_kv"], case["Dh"], case["P"], case["dtype"]
    s = dict(case=case, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if op == "norm_rope":
        T, Hq = case["T"], case["H_q"]
        slots, _, pages = _slots(case, g, T, 5)
        max_pos = 32768
        qkv = _randn(g, (T, Hq + 2 * H, D), dt)
        s |= dict(qkv=qkv, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], v=qkv[:, Hq + H:], slots=slots, cos_sin=_cos_sin(max_pos, D),
                  positions=torch.randint(0, max_pos, (T,), generator=g, device="cuda").to(torch.int32),
                  q_weight=1 + 0.1 * torch.randn(D, generator=g, device="cuda"),
                  k_weight=1 + 0.1 * torch.randn(D, generator=g, device="cuda"), eps=1e-6,
                  q_out=torch.zeros((T, Hq, D), dtype=DT[dt], device="cuda"),
                  k_pages=_randn(g, (pages, H, P, D), dt), v_pages=_randn(g, (pages, H, P, D), dt))
        return s
    if op == "int8_cache":
        T = case["T"]
        slots, used, pages = _slots(case, g, T, case["pages"] + 5)
        n = case["pages"]
        # a step's 64 tokens end 64 different sequences: one token on each of `pages` pages; a prompt fills its pages
        if T <= n:
            order = torch.randperm(pages, generator=g, device="cuda")[:n].to(torch.int32)
            off = torch.randint(0, P, (T,), generator=g, device="cuda")
            slots, used = (order[:T].long() * P + off).contiguous(), order
        codes = torch.randint(-127, 128, (2, pages, H, P, D), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
        s |= dict(k=_randn(g, (T, H, D), dt), v=_randn(g, (T, H, D), dt), slots=slots, src=used[:n].contiguous(),
                  dst=torch.randperm(n, generator=g, device="cuda").to(torch.int32), k_pages=codes[0].clone(),
                  v_pages=codes[1].clone(),
                  scales=torch.rand((pages, H, 2, P), generator=g, device="cuda") * 0.02 + 0.01,
                  k_out=torch.zeros((n, H, P, D), dtype=DT[dt], device="cuda"),
                  v_out=torch.zeros((n, H, P, D), dtype=DT[dt], device="cuda"))
        return s
    total, n = _lens(case)
    tab, pages = _table(case, g, total)
    rows, Hq = int(n.sum()), case["H_q"]
    s |= dict(tab=tab, lens=torch.from_numpy(total.astype(np.int32)).cuda(), scale=1.0 / math.sqrt(D),
              q=_randn(g, (rows, Hq, D), dt), out=torch.zeros((rows, Hq, D), dtype=torch.float32, device="cuda"),
              workspace=torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"))
    if op == "decode_int8":
        x = torch.randn((2, pages, H, P, D), generator=g, device="cuda")
        amax = x.abs().amax(-1)
        s |= dict(k_pages=torch.round(x[0] * (127.0 / amax[0])[..., None]).to(torch.int8),
                  v_pages=torch.round(x[1] * (127.0 / amax[1])[..., None]).to(torch.int8),
                  scales=(torch.stack([amax[0], amax[1]], 2) / 127.0).contiguous())
        return s
    b, pos, lo, hi, doc, start = _rows(case)
    s |= dict(k_pages=_randn(g, (pages, H, P, D), dt), v_pages=_randn(g, (pages, H, P, D), dt),
              key_start=torch.from_numpy(doc.astype(np.int32)).cuda() if case["docs"] else None,
              slopes=torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float() if case["alibi"] else None,
              q_start=torch.from_numpy(start.astype(np.int32)).cuda(), max_q=int(n.max()),
              prefix=torch.from_numpy(_prefix(case).astype(np.int32)).cuda() if case.get("prefix") else None)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, style):
    if style == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_norm_rope(s):
    c = s["case"]
    D, P = c["Dh"], c["P"]
    row = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = row[..., :D // 2], row[..., D // 2:]
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + s["eps"]) * s["q_weight"]
    k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + s["eps"]) * s["k_weight"]
    s["q_out"].copy_(_rotate(q, cos, sin, c["style"]))
    page, off = s["slots"] // P, s["slots"] % P
    s["k_pages"][page, :, off] = _rotate(k, cos, sin, c["style"]).to(s["k_pages"].dtype)
    s["v_pages"][page, :, off] = s["v"]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _quantise(x):
    x = x.float()
    amax = x.abs().amax(-1)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(x * inv[..., None]).to(torch.int8), amax / 127.0


def _plain_int8_cache(s):
    P = s["case"]["P"]
    page, off = s["slots"] // P, s["slots"] % P
    kc, ks = _quantise(s["k"])
    vc, vs = _quantise(s["v"])
    s["k_pages"][page, :, off] = kc
    s["v_pages"][page, :, off] = vc
    s["scales"][page, :, 0, off] = ks
    s["scales"][page, :, 1, off] = vs
    src, dst = s["src"].long(), s["dst"].long()
    s["k_out"][dst] = (s["k_pages"][src].float() * s["scales"][src, :, 0][..., None]).to(s["k_out"].dtype)
    s["v_out"][dst] = (s["v_pages"][src].float() * s["scales"][src, :, 1][..., None]).to(s["v_out"].dtype)
    return s["k_out"], s["v_out"], s["scales"]


def _gather(pages, tab):
    """[B, max_blocks] pages -> [B, H_kv, max_blocks * P, Dh] in 32 bits."""
    x = pages[tab.clamp(min=0).long()].float()
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s, q, k, v, seen, bias=None, cap=0.0):
    """q [B, H_kv, g * n, Dh], k / v [B, H_kv, T, Dh]; seen [B, 1, g * n, T]."""
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    if cap:
        x = cap * torch.tanh(x / cap)
    if bias is not None:
        x = x + bias
    x = torch.where(seen, x, torch.full((), -math.inf, device=x.device))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v)
    return torch.where(l > 0, o / l, torch.zeros_like(o))


def _plain_decode_int8(s):
    c = s["case"]
    B, H, D = c["B"], c["H_kv"], c["Dh"]
    tab = s["tab"].clamp(min=0).long()
    sc = s["scales"][tab]  # [B, max_blocks, H, 2, P]
    ks, vs = (sc[:, :, :, i].transpose(1, 2).flatten(2, 3)[..., None] for i in (0, 1))
    k, v = _gather(s["k_pages"], s["tab"]) * ks, _gather(s["v_pages"], s["tab"]) * vs
    t = torch.arange(k.shape[2], device="cuda")
    o = _attend(s, s["q"].float().view(B, H, -1, D), k, v, (t < s["lens"][:, None])[:, None, None, :])
    s["out"].copy_(o.reshape(s["out"].shape))
    return s["out"]


def _plain_mod(s):
    """Decode and chunked prefill: the rows of every sequence's chunk padded to the longest chunk."""
    c = s["case"]
    B, H, D, n = c["B"], c["H_kv"], c["Dh"], s["max_q"]
    g = c["H_q"] // H
    k, v = _gather(s["k_pages"], s["tab"]), _gather(s["v_pages"], s["tab"])
    i = torch.arange(n, device="cuda")
    qs, lens = s["q_start"].long(), s["lens"].long()
    cnt = qs[1:] - qs[:-1]
    row = qs[:-1, None] + i  # [B, n], rows behind a chunk are padding
    real = i < cnt[:, None]
    row = torch.where(real, row, torch.zeros_like(row))
    pos = (lens - cnt)[:, None] + i
    lo = torch.zeros_like(pos)
    if s["key_start"] is not None:
        lo = torch.maximum(lo, s["key_start"].long()[row])
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    hi = pos + 1
    if s["prefix"] is not None:
        hi = torch.maximum(hi, torch.minimum(s["prefix"].long(), lens)[:, None])
    t = torch.arange(k.shape[2], device="cuda")
    seen = (t >= lo[..., None]) & (t < hi[..., None]) & real[..., None]  # [B, n, T]
    seen = seen[:, None, None].expand(B, 1, g, n, -1).reshape(B, 1, g * n, -1)
    bias = None
    if s["slopes"] is not None:
        far = (pos[..., None] - t).abs().float()
        bias = -(s["slopes"].view(1, H, g, 1, 1) * far[:, None, None]).flatten(2, 3)
    q = s["q"].float()[row].view(B, n, H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, g * n, D)
    o = _attend(s, q, k, v, seen, bias, c["cap"])
    o = o.view(B, H, g, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H * g, D)
    s["out"].copy_(o[real])
    return s["out"]


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from paged_kv_cache_433_b200 import kvpaged as K

    c = s["case"]
    if c["op"] == "norm_rope":
        K.kv_norm_rope_append(s["k_pages"], s["v_pages"], s["k"], s["v"], s["slots"], s["positions"], s["cos_sin"],
                              s["k_weight"], s["eps"], c["P"], style=c["style"], q=s["q"], q_out=s["q_out"],
                              q_weight=s["q_weight"], err_flag=s["err"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if c["op"] == "int8_cache":
        K.kv_append_int8(s["k_pages"], s["v_pages"], s["scales"], s["k"], s["v"], s["slots"], c["P"], err_flag=s["err"])
        K.kv_dequant_pages_int8(s["k_out"], s["v_out"], s["k_pages"], s["v_pages"], s["scales"], s["src"], s["dst"],
                                err_flag=s["err"])
        return s["k_out"], s["v_out"], s["scales"]
    if c["op"] == "decode_int8":
        K.paged_decode_attention_int8(s["out"], s["q"], s["k_pages"], s["v_pages"], s["scales"], s["tab"], s["lens"],
                                      s["scale"], workspace=s["workspace"], err_flag=s["err"])
    elif c["op"] == "decode_mod":
        K.paged_decode_attention_mod(s["out"], s["q"], s["k_pages"], s["v_pages"], s["tab"], s["lens"], s["scale"],
                                     softcap=c["cap"], alibi_slopes=s["slopes"], window=c["window"],
                                     key_start=s["key_start"], workspace=s["workspace"], err_flag=s["err"])
    else:
        K.paged_prefill_attention_mod(s["out"], s["q"], s["q_start"], s["max_q"], s["k_pages"], s["v_pages"], s["tab"],
                                      s["lens"], s["scale"], softcap=c["cap"], alibi_slopes=s["slopes"],
                                      window=c["window"], key_start=s["key_start"], prefix_lens=s["prefix"],
                                      err_flag=s["err"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "int8_cache": _plain_int8_cache, "decode_int8": _plain_decode_int8,
            "decode_mod": _plain_mod, "prefill_mod": _plain_mod}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, H, D, P = case["op"], case["H_kv"], case["Dh"], case["P"]
    f8 = torch.float64
    if op == "norm_rope":
        half = D // 2
        ang = s["cos_sin"].to(f8)[s["positions"].long()]
        ix = torch.arange(half, device="cuda")
        ia, ib = (ix, ix + half) if case["style"] == "half" else (2 * ix, 2 * ix + 1)

        def turned(x, w):
            x = x.to(f8)
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + s["eps"]) * w.to(f8)
            y = torch.empty_like(x)
            co, si = ang[:, None, :half], ang[:, None, half:]
            y[..., ia] = x[..., ia] * co - x[..., ib] * si
            y[..., ib] = x[..., ib] * co + x[..., ia] * si
            return y

        kp, vp = s["k_pages"].to(f8), s["v_pages"].to(f8)
        flat = s["slots"]
        kp[flat // P, :, flat % P] = turned(s["k"], s["k_weight"])
        vp[flat // P, :, flat % P] = s["v"].to(f8)
        return turned(s["q"], s["q_weight"]), kp, vp
    if op == "int8_cache":
        # the code is defined by its two 32-bit roundings (of 127 / amax and of the product): made here from 64 bits
        outs, sc = [], s["scales"].to(f8)
        flat = s["slots"]
        for i, (new, pages) in enumerate(((s["k"], s["k_pages"]), (s["v"], s["v_pages"]))):
            x = new.to(f8)
            top = x.abs().max(-1).values
            inv = (127.0 / top).float().to(f8)
            code = (x * inv[..., None]).float().to(f8).round()
            val = pages.to(f8)
            val[flat // P, :, flat % P] = code
            sc[flat // P, :, i, flat % P] = top / 127.0
            o = torch.zeros((case["pages"], H, P, D), dtype=f8, device="cuda")
            o[s["dst"].long()] = val[s["src"].long()] * sc[s["src"].long(), :, i].unsqueeze(-1)
            outs.append(o)
        return outs[0], outs[1], sc
    total, n = _lens(case)
    out = torch.zeros(s["out"].shape, dtype=f8, device="cuda")
    g = case["H_q"] // H
    start = np.concatenate([[0], np.cumsum(n)])
    if op != "decode_int8":
        _, pos_all, lo_all, hi_all, _, _ = _rows(case)
    for b in range(case["B"]):
        L, r = int(total[b]), slice(int(start[b]), int(start[b + 1]))
        t = torch.arange(L, device="cuda")
        ids, off = s["tab"][b].long()[t // P], t % P
        k, v = s["k_pages"][ids, :, off].to(f8), s["v_pages"][ids, :, off].to(f8)  # [L, H, D]
        if op == "decode_int8":
            k = k * s["scales"][ids, :, 0, off].to(f8)[..., None]
            v = v * s["scales"][ids, :, 1, off].to(f8)[..., None]
        q = s["q"][r].to(f8)
        for h in range(case["H_q"]):
            x = (q[:, h] @ k[:, h // g].T) / math.sqrt(D)
            if op != "decode_int8":
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                p = torch.from_numpy(pos_all[r]).cuda()[:, None]
                if case["alibi"]:
                    x = x - s["slopes"][h].to(f8) * (p - t).abs()
                lo, hi = (torch.from_numpy(a[r]).cuda()[:, None] for a in (lo_all, hi_all))
                x = x.masked_fill((t < lo) | (t >= hi), -math.inf)
            w = torch.nan_to_num(torch.softmax(x, -1))
            out[r, h] = w @ v[:, h // g]
    return out
