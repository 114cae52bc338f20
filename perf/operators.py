"""Measured cases of the context operators: attention over packed prompts, single-token attention for a batch that
shares a long prefix, the append into that batch's cache, and eviction from it by accumulated attention weight.

A rollout of a long video (or the text side of a conditioning model) uses them in this order: the prompts of a batch
are attended in one packed call, their keys and values become a prefix that every sample of the batch shares, each new
step appends its tokens to the samples' own caches and attends prefix and cache together, adding up the weight that
each cached token receives, and a full cache is cut back to the tokens that received the most.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or, where ``own`` is set, by
the library's calls.  Ragged lengths are part of a case, as text, so that the work of a case is known without inputs.
"""
import math

import torch

own = False

DEV = "cuda"
NEG_INF = float("-inf")


def _text(values):
    return ",".join(str(int(v)) for v in values)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _ramp(n, lo, hi, turn=7):
    """n lengths spread over lo..hi, in an order that is neither rising nor falling."""
    return [lo + (hi - lo) * ((i * turn) % n) // max(1, n - 1) for i in range(n)]


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # Four short captions at once, every token seeing its whole caption: the call's latency.
        dict(name="packed_captions", op="packed", q_lens="17,1,40,5", k_lens="17,1,40,5", heads=4, kv_heads=2, dim=64, causal=False),
        # A batch of prompts of very different lengths, grouped heads.
        dict(name="packed_prompts", op="packed", q_lens=_text(_ramp(12, 100, 2500, 5)), k_lens=_text(_ramp(12, 100, 2500, 5)),
             heads=32, kv_heads=8, dim=128, causal=True),
        # One long token sequence at the small video workload's 12 heads, odd length, causal.
        dict(name="packed_long", op="packed", q_lens="16379", k_lens="16379", heads=12, kv_heads=12, dim=128, causal=True),
        # Prompts continued in pieces: new tokens against what is there already, a single token, a sequence without
        # new tokens, more tokens than keys (rows without any key).
        dict(name="packed_continued", op="packed", q_lens="256,1,0,130,511,64", k_lens="4352,777,33,60,2047,8000",
             heads=40, kv_heads=8, dim=128, causal=True),
        # Two samples, a short prefix: the latency of one step.
        dict(name="prefix_pair", op="prefix", steps=1, prefix=100, cap=64, lens="3,40", heads=4, kv_heads=2, dim=64, weights=False),
        # A batch that shares a system prompt, some hundred tokens of its own each.
        dict(name="prefix_batch", op="prefix", steps=1, prefix=8192, cap=1024, lens=_text(_ramp(32, 1, 1024, 5)),
             heads=32, kv_heads=8, dim=128, weights=False),
        # The largest: a long shared video context, many samples with long caches of their own.
        dict(name="prefix_large", op="prefix", steps=1, prefix=65531, cap=4096, lens=_text(_ramp(96, 500, 4096, 11)),
             heads=40, kv_heads=8, dim=128, weights=False),
        # Four tokens a step, every sample's weights summed up for a later eviction; one sample's cache is still empty
        # but for two of the four tokens.
        dict(name="prefix_weights", op="prefix", steps=4, prefix=1559, cap=6000, lens="2,4097," + _text(_ramp(14, 1800, 6000, 5)),
             heads=12, kv_heads=12, dim=128, weights=True),
        # The append of a step's token for a batch.
        dict(name="append_token", op="append", steps=1, cap=2048, lens=_text(_ramp(64, 0, 2047, 11)), kv_heads=8, dim=128),
        # The append of a whole latent frame (30 x 52 tokens) for a few samples.
        dict(name="append_frame", op="append", steps=1560, cap=8192, lens="0,1560,3121,6632", kv_heads=12, dim=128),
        # A small cache, cut a little; one sample is still below its budget.
        dict(name="evict_small", op="evict", cap=160, lens="150,90,101", budget=100, sinks=4, recent=16, kv_heads=2, dim=64),
        # Long caches cut to half.
        dict(name="evict_long", op="evict", cap=16384, lens=_text(_ramp(12, 9000, 16384, 5)), budget=8192, sinks=4, recent=1024,
             kv_heads=8, dim=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["packed", "packed", "packed", "prefix", "prefix", "prefix", "append", "evict"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 12])
    group = rng.choice([1, 1, 2, 3, 4, 5, 8])
    if op == "packed":
        while kv_heads * group > 40:
            group = rng.choice([1, 2, 3])
        longest = _log_int(rng, 4, 12000)
        # the plain form's scores, padded to the longest: at most 3e9 values
        most = max(1, int(3e9 / (longest * longest * kv_heads * group)))
        n = min(most, _log_int(rng, 1, 48))
        k_lens = [longest] + [_log_int(rng, 1, longest) for _ in range(n - 1)]
        rng.shuffle(k_lens)
        kind = rng.choice(["prompt", "prompt", "continued"])
        q_lens = k_lens if kind == "prompt" else [rng.choice([0, 1, rng.randint(1, k), min(k, 64), min(k + rng.randint(0, 9), longest)])
                                                  for k in k_lens]
        if not any(q_lens):
            q_lens = [1] * n
        return dict(op="packed", q_lens=_text(q_lens), k_lens=_text(k_lens), heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    causal=rng.random() < 0.75)
    if op == "prefix":
        cap = _log_int(rng, 16, 6000)
        steps = rng.choice([1, 1, 1, 2, 4, 5])
        n = min(_log_int(rng, 1, 96), max(1, int(1.2e9 / (cap * kv_heads * dim))))
        prefix = min(_log_int(rng, 1, 65531), max(1, int(4e8 / (n * steps * kv_heads * group))))
        lens = [rng.randint(min(steps, cap), cap) for _ in range(n)]
        return dict(op="prefix", steps=steps, prefix=prefix, cap=cap, lens=_text(lens), heads=kv_heads * group, kv_heads=kv_heads,
                    dim=dim, weights=rng.random() < 0.5)
    cap = _log_int(rng, 64, 16384)
    n = min(_log_int(rng, 1, 64), max(1, int(1e8 / (cap * kv_heads))), max(1, int(1.2e9 / (cap * kv_heads * dim))))
    if op == "append":
        steps = min(_log_int(rng, 1, 1560), cap)
        return dict(op="append", steps=steps, cap=cap, lens=_text(rng.randint(0, cap - steps) for _ in range(n)), kv_heads=kv_heads, dim=dim)
    budget = max(8, int(cap * rng.uniform(0.2, 0.9)))
    sinks = rng.randint(0, min(8, budget // 4))
    return dict(op="evict", cap=cap, lens=_text(rng.randint(1, cap) for _ in range(n)), budget=budget, sinks=sinks,
                recent=rng.randint(0, budget // 3), kv_heads=kv_heads, dim=dim)


# ------------------------------------------------------------------------------------------------ inputs


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _keys(g, heads_at, *shape):
    """Keys with a mean of their own for each head, as of tokens that many queries attend."""
    mean_shape = [1] * len(shape)
    mean_shape[heads_at], mean_shape[-1] = shape[heads_at], shape[-1]
    mean = 0.5 * torch.randn(mean_shape, generator=g, device=DEV)
    return (torch.randn(shape, generator=g, device=DEV) + mean).to(torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1009 + 17)
    s = dict(case)
    if case["op"] == "packed":
        ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
        tq, tk, hq, hk, d = sum(ql), sum(kl), case["heads"], case["kv_heads"], case["dim"]
        s["cu_q"] = _i32([sum(ql[:i]) for i in range(len(ql) + 1)])
        s["cu_k"] = _i32([sum(kl[:i]) for i in range(len(kl) + 1)])
        s["max_q"], s["max_k"] = max(ql), max(kl)
        s["q"], s["k"], s["v"] = _normal(g, tq, hq, d), _keys(g, 1, tk, hk, d), _normal(g, tk, hk, d)
        s["o"] = torch.empty((tq, hq, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((hq, tq), dtype=torch.float32, device=DEV)
        s["scale"] = d ** -0.5
        return s
    lens = _ints(case["lens"])
    b, hk, d, cap = len(lens), case["kv_heads"], case["dim"], case["cap"]
    s["lens_t"] = _i32(lens)
    s["k_cache"], s["v_cache"] = _keys(g, 1, b, hk, cap, d), _normal(g, b, hk, cap, d)
    # weight summed up over the steps so far: most tokens little, a few much, some none at all
    w = torch.exp(2.0 * torch.randn((b, hk, cap), generator=g, device=DEV))
    w = torch.where(torch.rand((b, hk, cap), generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
    if case["op"] == "prefix":
        t, hq, lp = case["steps"], case["heads"], case["prefix"]
        s["q"] = _normal(g, b, t, hq, d)
        s["prefix_k"], s["prefix_v"] = _keys(g, 1, lp, hk, d), _normal(g, lp, hk, d)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, hq, t), dtype=torch.float32, device=DEV)
        s["weight"] = w if case["weights"] else None
        s["scale"] = d ** -0.5
    elif case["op"] == "append":
        t = case["steps"]
        s["k_new"], s["v_new"] = _normal(g, b, t, hk, d), _normal(g, b, t, hk, d)
        s["weight"] = w
        s["lens_out"] = torch.zeros_like(s["lens_t"])
    else:
        s["weight"] = w
        s["k_out"], s["v_out"], s["weight_out"] = torch.zeros_like(s["k_cache"]), torch.zeros_like(s["v_cache"]), torch.zeros_like(w)
        s["lens_out"] = torch.zeros_like(s["lens_t"])
        s["kept"] = torch.zeros((b, hk, case["budget"]), dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ plain forms


def _softmax_parts(scores, seen):
    """exp(scores - max) where seen and the (max, sum) of each row; rows that see nothing get zeros and -inf."""
    scores = torch.where(seen, scores, NEG_INF)
    top = scores.amax(dim=-1, keepdim=True)
    e = torch.exp(scores - torch.where(top > NEG_INF, top, 0.0))
    return e, top.squeeze(-1), e.sum(dim=-1)


def _plain_packed(s):
    cu_q, cu_k, hq, hk, d = s["cu_q"].long(), s["cu_k"].long(), s["heads"], s["kv_heads"], s["dim"]
    ql, kl = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    qi, ki = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    # padded copies [sequences, heads, length, d]
    rows = (cu_q[:-1, None] + qi).clamp(max=s["q"].shape[0] - 1)
    cols = (cu_k[:-1, None] + ki).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][rows].float().reshape(len(ql), -1, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(len(ql), hk, -1, d)
    k, v = s["k"][cols].float().permute(0, 2, 1, 3), s["v"][cols].float().permute(0, 2, 1, 3)
    scores = ((q * s["scale"]) @ k.transpose(-1, -2)).reshape(len(ql), hq, s["max_q"], s["max_k"])
    seen = ki < kl[:, None, None]
    if s["causal"]:
        seen = seen & (ki <= qi[:, None] + (kl - ql)[:, None, None])
    e, top, total = _softmax_parts(scores, seen[:, None])
    del scores
    o = (e.reshape(len(ql), hk, -1, s["max_k"]) @ v).reshape(len(ql), hq, s["max_q"], d)
    o = o / torch.where(total > 0, total, 1.0)[..., None]
    lse = top + torch.log(total)
    real = qi < ql[:, None]
    s["o"] = o.permute(0, 2, 1, 3)[real].to(torch.bfloat16)
    s["lse"] = lse.permute(0, 2, 1)[real].transpose(0, 1).contiguous()
    return {"o": s["o"], "lse": s["lse"]}


def _plain_prefix(s):
    b, t, hq, d = s["q"].shape
    hk, cap, lp = s["kv_heads"], s["cap"], s["prefix"]
    q = s["q"].float().reshape(b, t, hk, hq // hk, d).permute(2, 0, 3, 1, 4) * s["scale"]          # [hk, b, group, t, d]
    pk, pv = s["prefix_k"].float().transpose(0, 1), s["prefix_v"].float().transpose(0, 1)           # [hk, lp, d]
    shared = (q.reshape(hk, -1, d) @ pk.transpose(-1, -2)).reshape(hk, b, -1, t, lp)
    ck, cv = s["k_cache"].float().transpose(0, 1), s["v_cache"].float().transpose(0, 1)             # [hk, b, cap, d]
    mine = (q.reshape(hk, b, -1, d) @ ck.transpose(-1, -2)).reshape(hk, b, -1, t, cap)
    last = s["lens_t"].long()[:, None] - t + torch.arange(t, device=DEV)                            # [b, t]
    seen = torch.arange(cap, device=DEV) <= last[..., None]
    e, top, total = _softmax_parts(torch.cat([shared, mine], dim=-1),
                                   torch.cat([seen.new_ones((b, t, lp)), seen], dim=-1)[:, None])
    del shared, mine
    o = (e[..., :lp].reshape(hk, -1, lp) @ pv).reshape(hk, b, -1, d) + e[..., lp:].reshape(hk, b, -1, cap) @ cv
    o = o.reshape(hk, b, -1, t, d) / total[..., None]
    s["o"] = o.permute(1, 3, 0, 2, 4).reshape(b, t, hq, d).to(torch.bfloat16)
    s["lse"] = (top + torch.log(total)).permute(1, 0, 2, 3).reshape(b, hq, t)
    out = {"o": s["o"], "lse": s["lse"]}
    if s["weight"] is not None:
        s["weight"] += (e[..., lp:] / total[..., None]).sum(dim=(2, 3)).transpose(0, 1)
        out["weight"] = s["weight"]
    return out


def _plain_append(s):
    b, t, hk, d = s["k_new"].shape
    at = s["lens_t"].long()[:, None] + torch.arange(t, device=DEV)
    seq = torch.arange(b, device=DEV)[:, None]
    s["k_cache"][seq, :, at] = s["k_new"]
    s["v_cache"][seq, :, at] = s["v_new"]
    s["weight"][seq, :, at] = 0.0
    s["lens_out"] = s["lens_t"] + t
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weight": s["weight"], "lens": s["lens_out"]}


def _plain_evict(s):
    cap, budget = s["cap"], s["budget"]
    n = s["lens_t"].long()[:, None, None]
    c = torch.arange(cap, device=DEV)
    rank = torch.where((c < s["sinks"]) | (c >= n - s["recent"]), float("inf"), s["weight"])
    rank = torch.where(c < n, rank, NEG_INF)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.sort(order, dim=-1).values
    place = torch.arange(budget, device=DEV)
    kept = torch.where(n <= budget, place, kept)
    count = torch.clamp(n, max=budget)
    live = (place < count)
    wide = live[..., None]
    source = kept[..., None].expand(-1, -1, -1, s["dim"])
    s["k_out"][:, :, :budget] = torch.where(wide, torch.gather(s["k_cache"], 2, source), s["k_out"][:, :, :budget])
    s["v_out"][:, :, :budget] = torch.where(wide, torch.gather(s["v_cache"], 2, source), s["v_out"][:, :, :budget])
    s["weight_out"][:, :, :budget] = torch.where(live, torch.gather(s["weight"], 2, kept), s["weight_out"][:, :, :budget])
    s["kept"] = torch.where(live, kept, -1).to(torch.int32)
    s["lens_out"] = count[:, 0, 0].to(torch.int32)
    return _evicted(s)


def _evicted(s):
    return {"k": s["k_out"], "v": s["v_out"], "weight": s["weight_out"], "lens": s["lens_out"], "kept": s["kept"]}


# ------------------------------------------------------------------------------------------------ the library's calls


def _own(s):
    import block_sparse_attention_lva_b200 as lva
    if s["op"] == "packed":
        lva.lva_packed_attn(s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"], s["cu_k"], s["scale"], causal=s["causal"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "prefix":
        if "workspace" not in s:
            b, t = s["q"].shape[:2]
            size = lva.lva_shared_prefix_workspace_bytes(b, t, s["heads"], s["kv_heads"], s["dim"], s["prefix"], s["cap"],
                                                         s["weight"] is not None)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        lva.lva_shared_prefix_attn(s["q"], s["prefix_k"], s["prefix_v"], s["k_cache"], s["v_cache"], s["lens_t"], s["o"], s["lse"],
                                   s["workspace"], s["scale"], weight=s["weight"])
        out = {"o": s["o"], "lse": s["lse"]}
        if s["weight"] is not None:
            out["weight"] = s["weight"]
        return out
    if s["op"] == "append":
        lva.lva_append_cache(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["weight"], s["lens_t"], s["lens_out"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weight": s["weight"], "lens": s["lens_out"]}
    lva.lva_evict_cache(s["k_cache"], s["v_cache"], s["weight"], s["lens_t"], s["k_out"], s["v_out"], s["weight_out"], s["lens_out"],
                        s["kept"], s["budget"], s["sinks"], s["recent"])
    return _evicted(s)


def run(state):
    if own:
        return _own(state)
    return {"packed": _plain_packed, "prefix": _plain_prefix, "append": _plain_append, "evict": _plain_evict}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ work and exact values


def _pairs(case, n_q, n_k):
    """Visible (query, key) pairs of one sequence."""
    if not case["causal"]:
        return n_q * n_k
    first = n_k - n_q + 1                     # keys that the first query sees (may be negative)
    lo = max(0, first)
    count = n_q - (lo - first)                # queries that see at least lo keys
    return count * (lo + n_k) // 2 if count > 0 else 0


def work(case):
    d = case["dim"]
    if case["op"] == "packed":
        ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
        pairs = sum(_pairs(case, a, b) for a, b in zip(ql, kl))
        rows = sum(ql) * case["heads"]
        return {"bytes": rows * (4 * d + 4) + sum(k for q, k in zip(ql, kl) if q) * case["kv_heads"] * 4 * d,
                "flops": 4 * d * case["heads"] * pairs}
    lens = _ints(case["lens"])
    b, hk = len(lens), case["kv_heads"]
    if case["op"] == "prefix":
        t, hq = case["steps"], case["heads"]
        seen = sum(max(0, n - t + 1 + i) for n in lens for i in range(t))
        live = sum(lens) * hk
        return {"bytes": b * t * hq * (4 * d + 4) + (case["prefix"] * hk + live) * 4 * d + (8 * live if case["weights"] else 0),
                "flops": 4 * d * hq * (b * t * case["prefix"] + seen)}
    if case["op"] == "append":
        return {"bytes": b * case["steps"] * hk * (8 * d + 4) + 8 * b, "flops": 0}
    kept = sum(min(n, case["budget"]) for n in lens) * hk
    ranked = sum(n for n in lens if n > case["budget"]) * hk
    return {"bytes": kept * (8 * d + 8) + 4 * ranked + 4 * b * hk * case["budget"], "flops": 0}


def _attend64(q, k, v, seen, scale):
    """q [h, n, d], k and v [h, m, d] in 64 bits, seen [n, m]: (o, lse, p)."""
    sc = torch.einsum("hnd,hmd->hnm", q, k) * scale
    sc.masked_fill_(~seen, NEG_INF)
    lse = torch.logsumexp(sc, dim=-1)
    p = torch.exp(sc - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("hnm,hmd->hnd", p, v), lse, p


def exact(case, seed):
    if case["op"] not in ("packed", "prefix"):
        return None
    s = prepare(case, seed)
    rep = case["heads"] // case["kv_heads"]
    wide = lambda x: x.double().transpose(0, 1).repeat_interleave(rep, dim=0)                        # noqa: E731
    if case["op"] == "packed":
        outs, lses = [], []
        at_q = at_k = 0
        for n, m in zip(_ints(case["q_lens"]), _ints(case["k_lens"])):
            k, v = wide(s["k"][at_k:at_k + m]), wide(s["v"][at_k:at_k + m])
            for r0 in range(0, n, 1024):
                r1 = min(n, r0 + 1024)
                limit = torch.arange(r0, r1, device=DEV)[:, None] + (m - n) if case["causal"] else m
                seen = (torch.arange(m, device=DEV)[None, :] <= limit).expand(r1 - r0, m)
                o, lse, _ = _attend64(s["q"][at_q + r0:at_q + r1].double().transpose(0, 1), k, v, seen, s["scale"])
                outs.append(o.transpose(0, 1))
                lses.append(lse)
            at_q, at_k = at_q + n, at_k + m
        return {"o": torch.cat(outs), "lse": torch.cat(lses, dim=1)}
    t, lp = case["steps"], case["prefix"]
    pk, pv = wide(s["prefix_k"]), wide(s["prefix_v"])
    os, lses = [], []
    weight = s["weight"].double() if s["weight"] is not None else None
    for i, n in enumerate(_ints(case["lens"])):
        k = torch.cat([pk, s["k_cache"][i, :, :n].double().repeat_interleave(rep, dim=0)], dim=1)
        v = torch.cat([pv, s["v_cache"][i, :, :n].double().repeat_interleave(rep, dim=0)], dim=1)
        limit = lp + n - t + torch.arange(t, device=DEV)[:, None]
        seen = (torch.arange(lp + n, device=DEV)[None, :] <= limit) | (torch.arange(lp + n, device=DEV) < lp)
        o, lse, p = _attend64(s["q"][i].double().transpose(0, 1), k, v, seen, s["scale"])
        os.append(o.transpose(0, 1))
        lses.append(lse)
        if weight is not None:
            weight[i, :, :n] += p[:, :, lp:].reshape(-1, rep * t, n).sum(dim=1)
    out = {"o": torch.stack(os), "lse": torch.stack(lses)}
    if weight is not None:
        out["weight"] = weight
    return out
