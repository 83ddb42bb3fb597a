"""The operators of the 8-bit KV cache, as a decode program calls them, and their plain forms.

The cache holds e4m3 codes [B, Hkv, capacity, d] with one power-of-two scale per block of 64 or 128
tokens and KV head (value = code * scale), a length per sequence, and per token and KV head the
attention weight it has received so far.  Five operators:

  append   new bf16 key / value rows are quantised into the cache at a position per sequence
  attn     attention of the newest query tokens over the whole cache, optionally adding each token's
           attention weight to the accumulated weights
  list     attention of one query token over an index list per query head (a selection's result)
  evict    the most recent tokens and those of the largest accumulated weight move to a smaller cache
  gather   the keys' dominant rotary dims as a compact bf16 copy (what a token selection reads)

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the framework's calls.
"""

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, heads_kv=8, group=4, head_dim=128, block=128, context=1024, ragged=False)
    c.update(kw)
    return c


def listed():
    return [
        # one token per sequence joins a batch's caches: every step of a served batch
        _case("append-step-b16", "append", batch=16, context=32768, n=1),
        # a whole prompt of one long request, right after its prefill
        _case("append-prompt-128k", "append", batch=1, context=0, n=131072),
        # a lone short conversation: latency is everything
        _case("attn-1k-b1", "attn", batch=1, context=1024, nq=1, weights=False),
        # an ordinary served batch at 32K
        _case("attn-32k-b16", "attn", batch=16, context=32768, nq=1, weights=False),
        # long contexts that will be evicted from: the weights are accumulated as well
        _case("attn-128k-b4-weights", "attn", batch=4, context=131072, nq=1, weights=True),
        # two tokens at once (a drafted token is checked), small heads and blocks, lengths all different
        _case("attn-ragged-8k-b24-d64", "attn", batch=24, context=8191, head_dim=64, block=64, ragged=True, nq=2,
              weights=True),
        # the decode step's focused attention: 256 selected tokens a query head
        _case("list-256-128k-b4", "list", batch=4, context=131072, k=256),
        # a larger, odd budget for many short sequences
        _case("list-1023-16k-b16", "list", batch=16, context=16383, k=1023, ragged=True),
        # a long prompt's cache shrunk to its budget
        _case("evict-128k-to-8k-b4", "evict", batch=4, context=131072, keep=8192, recent=1024),
        # the steady state: every hundred steps a budget cache is brought back to its budget
        _case("evict-2175-to-2048-b16", "evict", batch=16, context=2175, keep=2048, recent=128),
        # the compact keys of a whole long cache, once after the prompt
        _case("gather-128k-b4", "gather", batch=4, context=131072, nfc=12, npos=131072),
        # the compact key of the newest token, every step
        _case("gather-step-b16", "gather", batch=16, context=32768, nfc=12, npos=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(np.exp(rng.uniform(np.log(lo), np.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "list", "evict", "gather"])
    hkv, d, block = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]), rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 8])
    batch = _log_int(rng, 1, 64)
    budget = (4 * 8 * 131072 * 128) // (batch * hkv * d)  # tokens a sequence at the largest listed case
    context = _log_int(rng, 1, min(131072, budget))
    c = dict(op=op, batch=batch, heads_kv=hkv, group=group, head_dim=d, block=block, context=context,
             ragged=rng.random() < 0.5)
    if op == "append":
        c["n"] = _log_int(rng, 1, max(1, min(131072, budget // 4)))
        c["context"] = min(context, max(1, budget // 4))
    elif op == "attn":
        c["nq"] = _log_int(rng, 1, 16 // group)
        c["weights"] = rng.random() < 0.5
    elif op == "list":
        c["k"] = _log_int(rng, 1, max(1, min(2048, budget // group)))
    elif op == "evict":
        c["context"] = context = max(2, min(context, budget // 2))
        c["keep"] = _log_int(rng, 1, context)
        c["recent"] = rng.randint(0, c["keep"])
    else:
        c["nfc"] = 4 * rng.randint(1, d // 8)
        c["npos"] = _log_int(rng, 1, context)
        c["ragged"] = False
    return c


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------
def _cap(case):
    """Room for the context, what is appended, and some blocks to grow into."""
    return ((case["context"] + case.get("n", 0)) // 128 + 2) * 128


def prepare(case, seed):
    """Inputs from the seed alone: keys with a few strong dims (as rotated keys have), unit values."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, H, d, T, n = (case[k] for k in ("batch", "heads_kv", "head_dim", "block", "context"))
    cap = _cap(case)

    def rows(b, count, keys):
        x = torch.randn((b, H, count, d), generator=gen, device=dev)
        if keys:
            x[..., : d // 16] *= 3.0
        return x

    s = dict(case=case, cap=cap)
    s["k"] = torch.empty((B, H, cap, d), dtype=E4M3, device=dev)
    s["v"] = torch.empty_like(s["k"])
    s["k_scale"] = torch.empty((B, H, cap // T), device=dev)
    s["v_scale"] = torch.empty_like(s["k_scale"])
    for b in range(B):  # one sequence at a time: the 32-bit values need four times the cache's room
        for c, f, keys in (("k", "k_scale", True), ("v", "v_scale", False)):
            x = rows(1, cap, keys).view(1, H, cap // T, T, d)
            f_b = _scale(_need(x.abs().amax((-1, -2))))
            s[f][b] = f_b[0]
            s[c][b] = (x / f_b[..., None, None]).to(E4M3).view(H, cap, d)
    if case["ragged"]:
        s["lens"] = torch.randint(0, n + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        s["lens"][0] = n
    else:
        s["lens"] = torch.full((B,), n, dtype=torch.int32, device=dev)
    w = torch.rand((B, H, cap), generator=gen, device=dev)
    s["weight"] = torch.where(w < 0.05, torch.zeros_like(w), w ** 4 * 10.0)  # tokens never attended to tie at 0
    G, op = case["group"], case["op"]
    if op == "append":
        m = case["n"]
        s["K_new"] = rows(B, m, True).bfloat16()
        s["V_new"] = rows(B, m, False).bfloat16()
        s["at"] = s["lens"].clone()
        s["counts"] = (torch.randint(0, m + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
                       if case["ragged"] else torch.full((B,), m, dtype=torch.int32, device=dev))
    elif op == "attn":
        s["q"] = torch.randn((B, H * G, case["nq"], d), generator=gen, device=dev).bfloat16()
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:3], device=dev)
        s["weight_out"] = s["weight"].clone()
    elif op == "list":
        s["q"] = torch.randn((B, H * G, d), generator=gen, device=dev).bfloat16()
        k = case["k"]
        r = torch.rand((B, H * G, k), generator=gen, device=dev)
        lens = s["lens"][:, None, None]
        idx = (r * lens).to(torch.int32).clamp(max=(lens - 1).clamp(min=0)).sort(-1).values
        keep = torch.ones_like(idx, dtype=torch.bool)
        keep[..., 1:] = idx[..., 1:] != idx[..., :-1]
        idx = torch.where(keep & (lens > 0), idx, torch.full_like(idx, 1 << 30)).sort(-1).values
        s["idx"] = torch.where(idx == 1 << 30, torch.full_like(idx, -1), idx)  # ascending, -1 at the end
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device=dev)
    elif op == "evict":
        keep = case["keep"]
        dcap = (keep // 128 + 2) * 128
        s["dk"] = torch.zeros((B, H, dcap, d), dtype=E4M3, device=dev)
        s["dv"] = torch.zeros_like(s["dk"])
        s["dk_scale"] = torch.ones((B, H, dcap // T), device=dev)
        s["dv_scale"] = torch.ones_like(s["dk_scale"])
        s["dweight"] = torch.zeros((B, H, dcap), device=dev)
        s["dlens"] = torch.zeros((B,), dtype=torch.int32, device=dev)
        s["idx"] = torch.zeros((B, H, keep), dtype=torch.int32, device=dev)
    else:
        nfc = case["nfc"]
        pick = torch.rand((H, d // 2), generator=gen, device=dev).argsort(-1)[:, :nfc].sort(-1).values
        s["fc"] = pick.cpu().numpy().astype(np.int32)
        s["pairs"] = pick
        s["pos0"] = n - case["npos"]
        s["K_fc"] = torch.zeros((B, H, cap, 2 * nfc), dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _need(a):
    """The smallest e >= -126 with a <= 448 * 2^e (448 = 0.875 * 2^9), as int32."""
    m, e = torch.frexp(a)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(a > 0, e, torch.full_like(e, -126)).clamp(min=-126)


def _scale(e):
    """2^e for integers -126 <= e <= 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _exponent(scale):
    return (scale.view(torch.int32) >> 23) - 127


def _values(codes, scale, T):
    B, H, L, d = codes.shape
    return (codes.float().view(B, H, L // T, T, d) * scale[..., None, None]).view(B, H, L, d)


def _append_plain(s):
    T, n = s["case"]["block"], s["case"]["n"]
    at, counts = s["at"].long(), s["counts"].long()
    B, H, _, d = s["k"].shape
    nb = (n + T - 1) // T + 1  # blocks that n tokens from any position can touch
    dev = at.device
    blk = at[:, None] // T + torch.arange(nb, device=dev)
    row = (blk[..., None] * T + torch.arange(T, device=dev)).view(B, nb * T)
    end = (at + counts)[:, None]
    old, fresh = row < at[:, None], (row >= at[:, None]) & (row < end)
    src = (row - at[:, None]).clamp(0, n - 1)
    wide = (B, H, nb * T, d)
    at_row, at_src = row[:, None, :, None].expand(wide), src[:, None, :, None].expand(wide)
    at_blk = blk[:, None].expand(B, H, nb)
    old_b, fresh_b = (m.view(B, 1, nb, T).any(-1) for m in (old, fresh))
    blocks = lambda x: x.view(B, H, nb, T, d)  # noqa: E731
    for codes, scale, new in ((s["k"], s["k_scale"], s["K_new"]), (s["v"], s["v_scale"], s["V_new"])):
        x = new.float().gather(2, at_src)
        x = torch.where(torch.isfinite(x), x, torch.full_like(x, float("nan")))
        a = torch.where(fresh[:, None, :, None] & torch.isfinite(x), x.abs(), torch.zeros_like(x))
        was = scale.gather(2, at_blk)
        now = _scale(_need(blocks(a).amax((-1, -2))))
        now = torch.where(fresh_b, torch.where(old_b, torch.maximum(was, now), now), was)
        bits = codes.view(torch.uint8).gather(2, at_row)
        moved = blocks(bits.view(E4M3).float()) * (was / now)[..., None, None]
        put = torch.where(blocks(fresh[:, None, :, None].expand(wide)), blocks(x) / now[..., None, None], moved)
        put = put.to(E4M3).view(torch.uint8).view(wide)
        codes.view(torch.uint8).scatter_(2, at_row, torch.where((old | fresh)[:, None, :, None], put, bits))
        scale.scatter_(2, at_blk, now)
    at_w = row[:, None].expand(B, H, nb * T)
    w = s["weight"].gather(2, at_w)
    s["weight"].scatter_(2, at_w, torch.where(fresh[:, None], torch.zeros_like(w), w))
    s["lens"].copy_(end[:, 0])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "weight": s["weight"],
            "lens": s["lens"]}


def _softmax_plain(sc, seen):
    """Probabilities and log-sum-exp of the scores where `seen`; rows that see nothing give 0 and -inf."""
    sc = torch.where(seen, sc, torch.full_like(sc, float("-inf")))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(sc - m)
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    return p, (m + torch.log(total)).squeeze(-1)


def _attn_plain(s):
    c = s["case"]
    B, H, cap, d = s["k"].shape
    G, nq, n = c["group"], c["nq"], c["context"]
    n_up = -(-n // c["block"]) * c["block"]  # the blocks that hold anything
    nb = n_up // c["block"]
    k = _values(s["k"][:, :, :n_up], s["k_scale"][:, :, :nb], c["block"])
    q = s["q"].float().view(B, H, G * nq, d)
    sc = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    del k
    back = torch.arange(nq - 1, -1, -1, device=q.device).repeat(G)  # newer queries than this row's
    t = torch.arange(n_up, device=q.device)
    seen = t < (s["lens"][:, None, None, None] - back[None, None, :, None])
    p, lse = _softmax_plain(sc, seen)
    v = _values(s["v"][:, :, :n_up], s["v_scale"][:, :, :nb], c["block"])
    s["o"].copy_(torch.matmul(p, v).view_as(s["o"]))
    s["lse"].copy_(lse.view_as(s["lse"]))
    if not c["weights"]:
        return {"o": s["o"], "lse": s["lse"]}
    live = t < s["lens"][:, None, None]
    w = s["weight"][:, :, :n_up] + p.sum(2)
    s["weight_out"][:, :, :n_up] = torch.where(live, w, s["weight_out"][:, :, :n_up])
    return {"o": s["o"], "lse": s["lse"], "weight": s["weight_out"]}


def _list_plain(s):
    c = s["case"]
    B, H, cap, d = s["k"].shape
    G, k = c["group"], c["k"]
    idx = s["idx"].long().view(B, H, G * k)
    at = idx.clamp(min=0)
    wide = at[..., None].expand(B, H, G * k, d)

    def rows(codes, scale):
        r = codes.view(torch.uint8).gather(2, wide).view(E4M3).float()
        return (r * scale.gather(2, at // c["block"])[..., None]).view(B, H, G, k, d)

    q = s["q"].float().view(B, H, G, 1, d)
    sc = (q * rows(s["k"], s["k_scale"])).sum(-1) * d ** -0.5
    p, lse = _softmax_plain(sc, (idx >= 0).view(B, H, G, k))
    s["o"].copy_((p[..., None] * rows(s["v"], s["v_scale"])).sum(-2).view_as(s["o"]))
    s["lse"].copy_(lse.view_as(s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


def _evict_plain(s):
    c = s["case"]
    B, H, cap, d = s["k"].shape
    T, keep, recent = c["block"], c["keep"], c["recent"]
    t = torch.arange(cap, device=s["lens"].device)
    n = s["lens"].long()[:, None, None]
    # rank: the recent ones first, then by weight, then what is not there
    rank = torch.nan_to_num(s["weight"], nan=torch.finfo(torch.float32).max)
    rank = torch.where(t >= n - recent, torch.full_like(rank, float("inf")), rank)
    rank = torch.where(t < n, rank, torch.full_like(rank, float("-inf")))
    at = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    at = torch.where(at < n, at, torch.full_like(at, cap)).sort(-1).values
    there = at < cap
    s["idx"].copy_(torch.where(there, at, torch.full_like(at, -1)))
    at = at.clamp(max=cap - 1)
    nb = -(-keep // T)
    pad = nb * T - keep
    wide = at[..., None].expand(B, H, keep, d)
    for codes, scale, dst, dst_scale in ((s["k"], s["k_scale"], s["dk"], s["dk_scale"]),
                                         (s["v"], s["v_scale"], s["dv"], s["dv_scale"])):
        x = codes.view(torch.uint8).gather(2, wide).view(E4M3).float()
        e = _exponent(scale.gather(2, at // T))
        top = torch.where(torch.isfinite(x) & there[..., None], x.abs(), torch.zeros_like(x)).amax(-1)
        need = torch.where(top > 0, _need(top) + e, torch.full_like(e, -126)).clamp(min=-126)
        need = torch.nn.functional.pad(need, (0, pad), value=-126).view(B, H, nb, T).amax(-1)
        some = torch.nn.functional.pad(there, (0, pad)).view(B, H, nb, T).any(-1)
        by = (e - need.repeat_interleave(T, -1)[..., :keep]).clamp(-126, 127)
        put = (x * _scale(by)[..., None]).to(E4M3).view(torch.uint8)
        had = dst.view(torch.uint8)[:, :, :keep]
        dst.view(torch.uint8)[:, :, :keep] = torch.where(there[..., None], put, had)
        dst_scale[:, :, :nb] = torch.where(some, _scale(need), dst_scale[:, :, :nb])
    w = s["weight"].gather(2, at)
    s["dweight"][:, :, :keep] = torch.where(there, w, s["dweight"][:, :, :keep])
    s["dlens"].copy_(s["lens"].clamp(max=keep))
    return {"idx": s["idx"], "k": s["dk"], "v": s["dv"], "k_scale": s["dk_scale"], "v_scale": s["dv_scale"],
            "weight": s["dweight"], "lens": s["dlens"]}


def _gather_plain(s):
    c = s["case"]
    B, H, cap, d = s["k"].shape
    T, p0, m = c["block"], s["pos0"], c["npos"]
    dims = torch.cat([s["pairs"], s["pairs"] + d // 2], -1)
    x = s["k"][:, :, p0:p0 + m].view(torch.uint8).gather(3, dims[None, :, None, :].expand(B, H, m, dims.shape[-1]))
    f = s["k_scale"].gather(2, (torch.arange(p0, p0 + m, device=dims.device) // T).expand(B, H, m))
    s["K_fc"][:, :, p0:p0 + m] = (x.view(E4M3).float() * f[..., None]).to(torch.bfloat16)
    return {"K_fc": s["K_fc"]}


_PLAIN = {"append": _append_plain, "attn": _attn_plain, "list": _list_plain, "evict": _evict_plain,
          "gather": _gather_plain}


# ---------------------------------------------------------------------------------------------------
# The framework's calls.  A program makes its cache handle once and keeps it.
# ---------------------------------------------------------------------------------------------------
def _handle(s, prefix=""):
    from block_sparse_long_dual_b200 import sfa
    at = prefix + "cache"
    if at not in s:
        s[at] = sfa.KvCache8(k=s[prefix + "k"], v=s[prefix + "v"], k_scale=s[prefix + "k_scale"],
                             v_scale=s[prefix + "v_scale"], lens=s[prefix + "lens"], weight=s[prefix + "weight"],
                             block=s["case"]["block"])
    return s[at]


def _append_own(s):
    from block_sparse_long_dual_b200 import sfa
    sfa.cache8_append(_handle(s), s["K_new"], s["V_new"], at=s["at"], counts=s["counts"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "weight": s["weight"],
            "lens": s["lens"]}


def _attn_own(s):
    from block_sparse_long_dual_b200 import sfa
    cache, w = _handle(s), s["case"]["weights"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(sfa.cache8_attn_workspace(s["q"], cache, weights=w), dtype=torch.uint8,
                                     device=s["q"].device)
    sfa.cache8_attn(s["q"], cache, o=s["o"], lse=s["lse"], weight_in=s["weight"] if w else None,
                    weight_out=s["weight_out"] if w else None, workspace=s["workspace"])
    return {"o": s["o"], "lse": s["lse"], "weight": s["weight_out"]} if w else {"o": s["o"], "lse": s["lse"]}


def _list_own(s):
    from block_sparse_long_dual_b200 import sfa
    sfa.cache8_attn_list(s["q"], _handle(s), s["idx"], o=s["o"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


def _evict_own(s):
    from block_sparse_long_dual_b200 import sfa
    src, dst = _handle(s), _handle(s, "d")
    if "workspace" not in s:
        s["workspace"] = torch.empty(sfa.cache8_evict_workspace(src, s["case"]["keep"]), dtype=torch.uint8,
                                     device=s["k"].device)
    sfa.cache8_evict(src, dst, keep=s["case"]["keep"], recent=s["case"]["recent"], idx=s["idx"],
                     workspace=s["workspace"])
    return {"idx": s["idx"], "k": s["dk"], "v": s["dv"], "k_scale": s["dk_scale"], "v_scale": s["dv_scale"],
            "weight": s["dweight"], "lens": s["dlens"]}


def _gather_own(s):
    from block_sparse_long_dual_b200 import sfa
    sfa.cache8_fc_gather(_handle(s), s["fc"], K_fc=s["K_fc"], pos0=s["pos0"], npos=s["case"]["npos"])
    return {"K_fc": s["K_fc"]}


_OWN = {"append": _append_own, "attn": _attn_own, "list": _list_own, "evict": _evict_own, "gather": _gather_own}


# ---------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------
def work(case):
    B, H, G, d, T, n = (case[k] for k in ("batch", "heads_kv", "group", "head_dim", "block", "context"))
    heads = B * H
    if case["ragged"]:
        n = (n + 1) // 2 if B > 1 else n  # lengths spread evenly over [0, n]
    op = case["op"]
    if op == "append":
        m = case["n"] // 2 + 1 if case["ragged"] else case["n"]
        return {"bytes": heads * m * (2 * d * 2 + 2 * d + 4 + 16 / T), "flops": heads * m * 2 * d * 2}
    if op == "attn":
        rows = G * case["nq"]
        b = heads * (n * (2 * d + 8 / T + (8 if case["weights"] else 0)) + rows * (4 * d + 4))
        return {"bytes": b, "flops": heads * n * rows * 4 * d}
    if op == "list":
        k = min(case["k"], max(n, 1))
        return {"bytes": heads * G * (k * (2 * d + 4 + 8) + 4 * d + 4), "flops": heads * G * k * 4 * d}
    if op == "evict":
        k = min(case["keep"], n)
        return {"bytes": heads * (4 * n + k * (2 * 2 * d + 8 + 4 + 16 / T)), "flops": heads * (n + k * 2 * d)}
    return {"bytes": heads * case["npos"] * (2 * case["nfc"] + 4 * case["nfc"] + 4 / T), "flops": heads * case["npos"] * 2 * case["nfc"]}


# ---------------------------------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------------------
def _e4m3_64(x):
    """x rounded to the nearest e4m3 value, ties to even: 3 fraction bits, exponents from -6 up."""
    e = torch.frexp(x).exponent - 1
    step = torch.exp2((e.clamp(min=-6) - 3).double())
    return torch.round(x / step) * step


def _block_scale_64(a):
    """The smallest 2^e >= 2^-126 with a <= 448 * 2^e."""
    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e)
    e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e)
    return torch.exp2(torch.where(a > 0, e, torch.full_like(e, -126.0)).clamp(min=-126.0))


def _exact_append(s):
    c, T = s["case"], s["case"]["block"]
    out = {}
    for name, new in (("k", s["K_new"]), ("v", s["V_new"])):
        codes, scale = s[name].double(), s[name + "_scale"].double()
        for b in range(c["batch"]):
            a, m = int(s["at"][b]), int(s["counts"][b])
            if m == 0:
                continue
            for h in range(c["heads_kv"]):
                x = new[b, h, :m].double()
                first, last = a // T, (a + m - 1) // T
                top = torch.zeros(((last - first + 1) * T,), dtype=torch.float64, device=x.device)
                top[a - first * T: a - first * T + m] = x.abs().amax(-1)
                f = _block_scale_64(top.view(-1, T).amax(-1))
                if a % T:
                    was = scale[b, h, first].clone()
                    f[0] = torch.maximum(f[0], was)
                    codes[b, h, first * T: a] = _e4m3_64(codes[b, h, first * T: a] * (was / f[0]))
                scale[b, h, first: last + 1] = f
                per = f.repeat_interleave(T)[a - first * T: a - first * T + m]
                codes[b, h, a: a + m] = _e4m3_64(x / per[:, None])
        out[name], out[name + "_scale"] = codes, scale
    w = s["weight"].double()
    for b in range(c["batch"]):
        w[b, :, int(s["at"][b]): int(s["at"][b] + s["counts"][b])] = 0
    return {**out, "weight": w, "lens": s["at"] + s["counts"]}


def _exact_attn(s):
    c, T = s["case"], s["case"]["block"]
    B, H, G, nq, d = c["batch"], c["heads_kv"], c["group"], c["nq"], c["head_dim"]
    o = torch.zeros((B, H, G, nq, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, H, G, nq), float("-inf"), dtype=torch.float64, device=o.device)
    w = s["weight_out"].double()
    q = s["q"].double().view(B, H, G, nq, d)
    for b in range(B):
        n = int(s["lens"][b])
        if n == 0:
            continue
        w[b, :, :n] = s["weight"][b, :, :n].double()
        f = [s[x][b].double().repeat_interleave(T, -1)[:, :n, None] for x in ("k_scale", "v_scale")]
        k, v = s["k"][b, :, :n].double() * f[0], s["v"][b, :, :n].double() * f[1]
        for i in range(nq):
            m = n - (nq - 1 - i)
            if m <= 0:
                continue
            sc = torch.einsum("hgd,htd->hgt", q[b, :, :, i], k[:, :m]) / d ** 0.5
            lse[b, :, :, i] = torch.logsumexp(sc, -1)
            p = torch.softmax(sc, -1)
            o[b, :, :, i] = torch.einsum("hgt,htd->hgd", p, v[:, :m])
            w[b, :, :m] += p.sum(1)
    out = {"o": o.view(B, H * G, nq, d), "lse": lse.view(B, H * G, nq)}
    return {**out, "weight": w} if c["weights"] else out


def _exact_list(s):
    c, T = s["case"], s["case"]["block"]
    B, H, G, d = c["batch"], c["heads_kv"], c["group"], c["head_dim"]
    o = torch.zeros((B, H * G, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, H * G), float("-inf"), dtype=torch.float64, device=o.device)
    count = (s["idx"] >= 0).sum(-1).tolist()  # ascending, the -1 at the end
    for b in range(B):
        for r in range(H * G):
            if count[b][r] == 0:
                continue
            t = s["idx"][b, r, : count[b][r]].long()
            k = s["k"][b, r // G][t].double() * s["k_scale"][b, r // G][t // T].double()[:, None]
            v = s["v"][b, r // G][t].double() * s["v_scale"][b, r // G][t // T].double()[:, None]
            sc = (k @ s["q"][b, r].double()) / d ** 0.5
            lse[b, r] = torch.logsumexp(sc, 0)
            o[b, r] = torch.softmax(sc, 0) @ v
    return {"o": o, "lse": lse}


def _exact_evict(s):
    c, T = s["case"], s["case"]["block"]
    B, H, keep, recent = c["batch"], c["heads_kv"], c["keep"], c["recent"]
    out = {"idx": torch.full((B, H, keep), -1, dtype=torch.int32, device=s["k"].device),
           "weight": s["dweight"].double(), "lens": s["lens"].clamp(max=keep)}
    for name in ("k", "v"):
        out[name], out[name + "_scale"] = s["d" + name].double(), s["d" + name + "_scale"].double()
    weight = s["weight"].double().cpu().numpy()
    for b in range(B):
        n = int(s["lens"][b])
        for h in range(H):
            if n <= keep:
                t = np.arange(n)
            else:
                old = weight[b, h, : n - recent]
                best = np.lexsort((np.arange(len(old)), -old))[: keep - recent]
                t = np.sort(np.concatenate([best, np.arange(n - recent, n)]))
            if len(t) == 0:
                continue
            t = torch.from_numpy(t).to(s["k"].device)
            out["idx"][b, h, : len(t)] = t.int()
            out["weight"][b, h, : len(t)] = s["weight"][b, h][t].double()
            nb = -(-len(t) // T)
            for name in ("k", "v"):
                x = s[name][b, h][t].double() * s[name + "_scale"][b, h][t // T].double()[:, None]
                top = torch.zeros((nb * T,), dtype=torch.float64, device=x.device)
                top[: len(t)] = x.abs().amax(-1)
                f = _block_scale_64(top.view(nb, T).amax(-1))
                out[name + "_scale"][b, h, :nb] = f
                out[name][b, h, : len(t)] = _e4m3_64(x / f.repeat_interleave(T)[: len(t), None])
    return out


def _exact_gather(s):
    c, T = s["case"], s["case"]["block"]
    d, p0, m = c["head_dim"], s["pos0"], c["npos"]
    out = s["K_fc"].double()
    for h in range(c["heads_kv"]):
        for j, pair in enumerate(s["fc"][h].tolist()):
            for col, dim in ((j, pair), (c["nfc"] + j, pair + d // 2)):
                f = s["k_scale"][:, h].double().repeat_interleave(T, -1)[:, p0:p0 + m]
                out[:, h, p0:p0 + m, col] = s["k"][:, h, p0:p0 + m, dim].double() * f
    return {"K_fc": out}


_EXACT = {"append": _exact_append, "attn": _exact_attn, "list": _exact_list, "evict": _exact_evict,
          "gather": _exact_gather}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
