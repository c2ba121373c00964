"""Cases for the serving operators around the paged cache: appending rotated
keys and values, attention of new tokens over the paged cache, and attention
over whole packed prompts.

``own`` false: the operators in plain torch, in 32 bits, rounded once at the
end.  ``own`` true: the framework's calls.  All three take packed tokens:
sequence b of a batch holds the tokens cu[b] .. cu[b + 1] - 1.
"""
import math
import random

import torch

own = False

# head layouts of the repository's workloads: (Hq, Hkv, D)
TINY, LLAMA8B, LLAMA70B, D64 = (8, 2, 64), (32, 8, 128), (64, 8, 128), (32, 8, 64)


def _heads(h):
    return {"Hq": h[0], "Hkv": h[1], "D": h[2]}


def listed():
    return [
        # ---- append: one decode step's tokens (latency)
        dict(name="append_decode_b16", op="append", B=16, chunks=0, n_lo=1, n_hi=1, ctx_lo=500, ctx_hi=4096, P=16,
             rot=128, interleaved=False, sizes=1, **_heads(LLAMA8B)),
        # a mixed serving batch: 8 prompt chunks between 56 decode tokens, 64-token pages, half of each head rotated
        dict(name="append_mixed_b64", op="append", B=64, chunks=8, n_lo=100, n_hi=512, ctx_lo=0, ctx_hi=2048, P=64,
             rot=64, interleaved=True, sizes=2, **_heads(LLAMA70B)),
        # four whole prompts entering an empty cache (bandwidth)
        dict(name="append_prompts_8k", op="append", B=4, chunks=4, n_lo=1900, n_hi=2200, ctx_lo=0, ctx_hi=0, P=16,
             rot=128, interleaved=False, sizes=3, **_heads(LLAMA8B)),
        # ---- chunk: a single token of one short sequence (latency)
        dict(name="chunk_decode_b1_l2048", op="chunk", B=1, chunks=0, n_lo=1, n_hi=1, ctx_lo=2047, ctx_hi=2047, P=16,
             window=0, sizes=4, **_heads(TINY)),
        # a decode step over the whole cache of 16 sequences (cache bandwidth)
        dict(name="chunk_decode_b16_l32768", op="chunk", B=16, chunks=0, n_lo=1, n_hi=1, ctx_lo=32767, ctx_hi=32767,
             P=16, window=0, sizes=5, **_heads(LLAMA8B)),
        # verification of 2 to 8 draft tokens over ragged contexts
        dict(name="chunk_verify_b24", op="chunk", B=24, chunks=24, n_lo=2, n_hi=8, ctx_lo=900, ctx_hi=16384, P=64,
             window=0, sizes=6, **_heads(LLAMA70B)),
        # a mixed serving batch: 3 prompt chunks between 13 decode tokens
        dict(name="chunk_mixed_b16", op="chunk", B=16, chunks=3, n_lo=200, n_hi=512, ctx_lo=100, ctx_hi=8000, P=16,
             window=0, sizes=7, **_heads(LLAMA8B)),
        # one 2048-token chunk of a long prompt (tensor rate)
        dict(name="chunk_prefill_c2048", op="chunk", B=1, chunks=1, n_lo=2048, n_hi=2048, ctx_lo=30720, ctx_hi=30720,
             P=64, window=0, sizes=8, **_heads(LLAMA8B)),
        # ---- prompt: a few short requests (latency)
        dict(name="prompt_short_b4", op="prompt", B=4, chunks=4, n_lo=37, n_hi=300, ctx_lo=0, ctx_hi=0, P=0, window=0,
             sizes=9, **_heads(TINY)),
        # packed prompts of different lengths
        dict(name="prompt_packed_b12", op="prompt", B=12, chunks=12, n_lo=150, n_hi=2048, ctx_lo=0, ctx_hi=0, P=0,
             window=0, sizes=10, **_heads(LLAMA8B)),
        # one long prompt (tensor rate)
        dict(name="prompt_8192", op="prompt", B=1, chunks=1, n_lo=8192, n_hi=8192, ctx_lo=0, ctx_hi=0, P=0, window=0,
             sizes=11, **_heads(LLAMA8B)),
        # long prompts through a sliding-window layer, 64-wide heads
        dict(name="prompt_window_b2", op="prompt", B=2, chunks=2, n_lo=4000, n_hi=5000, ctx_lo=0, ctx_hi=0, P=0,
             window=1024, sizes=12, **_heads(D64)),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        op = rng.choice(("append", "chunk", "prompt"))
        c = dict(op=op, sizes=rng.randrange(1 << 20))
        hkv = rng.choice((1, 2, 4, 8))
        c.update(Hq=hkv * rng.choice((1, 2, 3, 4, 5, 7, 8)), Hkv=hkv, D=rng.choice((64, 128, 128)))
        B = _log(rng, 1, 64)
        if op == "prompt":
            lo = _log(rng, 1, 4096)
            c.update(B=B, chunks=B, n_lo=lo, n_hi=_log(rng, lo, 8192), ctx_lo=0, ctx_hi=0, P=0,
                     window=rng.choice((0, 0, _log(rng, 1, 4096))))
        else:
            lo = _log(rng, 1, 1024)
            ctx = rng.choice((0, _log(rng, 1, 16384)))
            c.update(B=B, chunks=rng.choice((0, B, rng.randint(0, B))), n_lo=lo, n_hi=_log(rng, lo, 2048), ctx_lo=ctx,
                     ctx_hi=_log(rng, max(ctx, 1), 32768), P=rng.choice((16, 32, 48, 64, 128)))
            if op == "append":
                c.update(rot=rng.choice((c["D"], c["D"] // 2)), interleaved=rng.choice((False, True)))
            else:
                c.update(window=rng.choice((0, 0, _log(rng, 1, 8192))))
        n, ctx = _lens(c)
        rows, keys = c["B"] * c["Hq"] * max(n), max(a + b for a, b in zip(n, ctx))
        if op == "append":
            fits = sum(n) <= 8192 and c["B"] * keys * c["Hkv"] * c["D"] <= 1 << 28
        else:
            fits = rows * keys <= 1 << 31 and c["B"] * keys * c["Hkv"] * c["D"] <= 1 << 29
        w = work(c)
        if fits and w["bytes"] >= 50_000 and w["bytes"] <= 2.1e9 and w["flops"] <= 1.0e12:
            return c


def _lens(case):
    """(new tokens, tokens cached before) of each sequence: from the case alone."""
    r = random.Random(case["sizes"])
    n = [r.randint(case["n_lo"], case["n_hi"]) if i < case["chunks"] else 1 for i in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    order = list(range(case["B"]))
    r.shuffle(order)
    return [n[i] for i in order], ctx


def _bf16(shape, g):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, ctx = _lens(case)
    B, Hq, Hkv, D, P = (case[k] for k in ("B", "Hq", "Hkv", "D", "P"))
    total = sum(n)
    s = dict(case=case, n=torch.tensor(n, device="cuda", dtype=torch.int32), max_n=max(n), total=total)
    s["cu"] = torch.tensor([sum(n[:i]) for i in range(B + 1)], device="cuda", dtype=torch.int32)
    s["q"] = _bf16((total, Hq, D), g)
    if case["op"] == "prompt":
        s.update(k=_bf16((total, Hkv, D), g), v=_bf16((total, Hkv, D), g), max_len=max(n),
                 scale=1.0 / math.sqrt(D), o=torch.empty_like(s["q"]), lse=torch.empty((total, Hq), device="cuda"))
        return s
    end = [a + b for a, b in zip(n, ctx)]
    pages = [-(-e // P) for e in end]
    pool, width = sum(pages) + 2, max(pages)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = torch.tensor([sum(pages[:i]) for i in range(B)], device="cuda")
    at = (first[:, None] + col[None, :]).clamp_(max=pool - 1)
    used = col[None, :] < torch.tensor(pages, device="cuda")[:, None]
    s["page_table"] = torch.where(used, perm[at], torch.full_like(perm[at], -1)).contiguous()
    s["k_cache"], s["v_cache"] = _bf16((pool, Hkv, P, D), g), _bf16((pool, Hkv, P, D), g)
    s["max_len"] = max(end)
    if case["op"] == "chunk":
        s.update(seq_lens=torch.tensor(end, device="cuda", dtype=torch.int32), scale=1.0 / math.sqrt(D),
                 o=torch.empty_like(s["q"]), lse=torch.empty((total, Hq), device="cuda"))
        return s
    rot = case["rot"]
    freq = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(max(end), device="cuda", dtype=torch.float64)[:, None] * freq[None, :]
    s.update(k=_bf16((total, Hkv, D), g), v=_bf16((total, Hkv, D), g),
             rope=torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32).contiguous(),
             seq_lens=torch.tensor(ctx, device="cuda", dtype=torch.int32),
             summaries=_bf16((pool, Hkv, D), g), q_out=torch.empty_like(s["q"]),
             new_lens=torch.empty(B, device="cuda", dtype=torch.int32))
    return s


# ------------------------------------------------------------------ plain forms
def _tokens(s):
    """(sequence, index within the sequence's new tokens) of every packed token"""
    b = torch.repeat_interleave(torch.arange(len(s["n"]), device="cuda"), s["n"].long(), output_size=s["total"])
    return b, torch.arange(s["total"], device="cuda") - s["cu"].long()[b]


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] bf16, cos / sin [T, r / 2] -> rotated, rounded to bf16 once"""
    r2 = cos.shape[1]
    x = x.float()
    c, s = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:2 * r2:2], x[..., 1:2 * r2:2]) if interleaved else (x[..., :r2], x[..., r2:2 * r2])
    ra, rb = a * c - b * s, b * c + a * s
    head = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((head, x[..., 2 * r2:]), -1).to(torch.bfloat16)


def _append(s):
    case, P = s["case"], s["case"]["P"]
    b, i = _tokens(s)
    pos = s["seq_lens"].long()[b] + i
    r2 = case["rot"] // 2
    cos, sin = s["rope"][pos, :r2], s["rope"][pos, r2:]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, case["interleaved"]))
    page = s["page_table"].long()[b, pos // P]
    s["k_cache"][page, :, pos % P] = _rotate(s["k"], cos, sin, case["interleaved"])
    s["v_cache"][page, :, pos % P] = s["v"]
    new = s["seq_lens"] + s["n"]
    valid = (new.long()[b] - pos // P * P).clamp(max=P)
    keys = s["k_cache"][page].float()
    keys = keys.masked_fill_((torch.arange(P, device="cuda")[None, :] >= valid[:, None])[:, None, :, None], 0.0)
    s["summaries"][page] = (keys.sum(2) / valid[:, None, None]).to(torch.bfloat16)
    s["new_lens"].copy_(new)
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache", "summaries", "new_lens")}


def _attend(s, k, v, lens, window):
    """k, v [B, Hkv, L, D] in 32 bits, padded; lens [B]"""
    B, Hkv, L, D = k.shape
    Hq, N = s["q"].shape[1], s["max_n"]
    b, i = _tokens(s)
    q = torch.zeros((B, N, Hq, D), device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, Hq // Hkv, N, L)
    at = (lens - s["n"]).long()[:, None] + torch.arange(N, device="cuda")[None, :]
    j = torch.arange(L, device="cuda")
    seen = (j <= at[..., None]) & (j < lens.long()[:, None, None])
    if window:
        seen &= j > at[..., None] - window
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, L), v).view(B, Hkv, Hq // Hkv, N, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    lse = (m + z.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[b, i]
    s["o"].copy_(o.to(torch.bfloat16))
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(B, N, Hq)[b, i])
    return s["o"], s["lse"]


def _chunk(s):
    L = s["max_len"]
    pages = s["page_table"].long().clamp(min=0)
    k, v = (s[x][pages].permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :L].float() for x in ("k_cache", "v_cache"))
    return _attend(s, k, v, s["seq_lens"], s["case"]["window"])


def _prompt(s):
    at = (s["cu"].long()[:-1, None] + torch.arange(s["max_len"], device="cuda")[None, :]).clamp_(max=s["total"] - 1)
    k, v = (s[x][at].transpose(1, 2).float() for x in ("k", "v"))
    return _attend(s, k, v, s["n"], s["case"]["window"])


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _append, "chunk": _chunk, "prompt": _prompt}[op](s)
    import paged_sparse_kv_sa_b200 as sa

    if op == "append":
        sa.sa_append_kv_rope(s["q"], s["k"], s["v"], s["cu"], s["rope"], s["k_cache"], s["v_cache"], s["page_table"],
                             s["seq_lens"], s["summaries"], interleaved=s["case"]["interleaved"], q_out=s["q_out"],
                             out_seq_lens=s["new_lens"])
        return {k: s[k] for k in ("q_out", "k_cache", "v_cache", "summaries", "new_lens")}
    if "workspace" not in s:   # kept from pass to pass, as a serving loop keeps it
        s["workspace"] = sa.dense_attention_workspace(s["total"], s["q"].shape[1], s["case"]["Hkv"], s["case"]["D"],
                                                      s["q"].device)
    if op == "chunk":
        return sa.sa_chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"], s["cu"],
                                     s["scale"], window=s["case"]["window"], o_out=s["o"], lse_out=s["lse"],
                                     workspace=s["workspace"])
    return sa.sa_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["cu"], s["scale"], window=s["case"]["window"],
                                  o_out=s["o"], lse_out=s["lse"], workspace=s["workspace"])


# ------------------------------------------------------------------ work and exact values
def work(case):
    n, ctx = _lens(case)
    Hq, Hkv, D, P = (case[k] for k in ("Hq", "Hkv", "D", "P"))
    total = sum(n)
    if case["op"] == "append":
        # queries and new keys and values in and out, the table's rows, the keys already in the pages that grow, and
        # their summaries
        old = sum(c % P for c in ctx)
        touched = sum((c + m - 1) // P - c // P + 1 for c, m in zip(ctx, n))
        by = total * (2 * Hq + 4 * Hkv) * D * 2 + total * case["rot"] * 4 + (old + touched) * Hkv * D * 2
        return {"bytes": by, "flops": total * (Hq + Hkv) * case["rot"] * 3}
    keys = pairs = 0
    for m, c in zip(n, ctx):
        w = case["window"] or m + c
        keys += min(m + c, w + m - 1)
        # visible keys of the tokens at positions c .. c + m - 1: min(position + 1, w)
        grow = max(0, min(m, w - c))
        pairs += grow * (2 * c + grow + 1) // 2 + (m - grow) * w
    by = total * Hq * (2 * D * 2 + 4) + keys * Hkv * 2 * D * 2
    return {"bytes": by, "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    """From the definitions, in 64 bits, a sequence and a kv head at a time."""
    s = prepare(case, seed)
    n, ctx = _lens(case)
    Hq, Hkv, D, P = (case[k] for k in ("Hq", "Hkv", "D", "P"))
    G = Hq // Hkv
    if case["op"] == "append":
        out = {k: s[k].double() for k in ("q", "k_cache", "v_cache", "summaries")}
        for b, (m, c) in enumerate(zip(n, ctx)):
            a = int(s["cu"][b])
            r2 = case["rot"] // 2
            z = torch.complex(s["rope"][c:c + m, :r2].double(), s["rope"][c:c + m, r2:].double())[:, None, :]
            turned = []
            for x in (s["q"][a:a + m].double(), s["k"][a:a + m].double()):
                re, im = (slice(0, 2 * r2, 2), slice(1, 2 * r2, 2)) if case["interleaved"] else (slice(0, r2), slice(r2, 2 * r2))
                w = torch.complex(x[..., re], x[..., im]) * z
                x[..., re], x[..., im] = w.real, w.imag
                turned.append(x)
            out["q"][a:a + m] = turned[0]
            for p in range(c // P, (c + m - 1) // P + 1):
                ph = int(s["page_table"][b, p])
                lo, hi = max(c, p * P), min(c + m, p * P + P)
                out["k_cache"][ph][:, lo - p * P:hi - p * P] = turned[1][lo - c:hi - c].transpose(0, 1)
                out["v_cache"][ph][:, lo - p * P:hi - p * P] = s["v"][a + lo - c:a + hi - c].double().transpose(0, 1)
                out["summaries"][ph] = out["k_cache"][ph][:, :hi - p * P].mean(1)
        return {"q_out": out["q"], "k_cache": out["k_cache"], "v_cache": out["v_cache"],
                "summaries": out["summaries"], "new_lens": s["seq_lens"] + s["n"]}
    o = torch.zeros((s["total"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], Hq), dtype=torch.float64, device="cuda")
    for b, (m, c) in enumerate(zip(n, ctx)):
        a, L = int(s["cu"][b]), m + c
        if case["op"] == "chunk":
            ph = s["page_table"][b, :-(-L // P)].long()
        hidden = torch.ones((m, L), dtype=torch.bool, device="cuda").tril(c)
        if case["window"]:
            hidden &= ~torch.ones_like(hidden).tril(c - case["window"])
        hidden = ~hidden
        for h in range(Hkv):
            if case["op"] == "chunk":
                k, v = (s[x][ph, h].reshape(-1, D)[:L].double() for x in ("k_cache", "v_cache"))
            else:
                k, v = (s[x][a:a + m, h].double() for x in ("k", "v"))
            for i in range(h * G, h * G + G):
                x = (s["q"][a:a + m, i].double() @ k.T) * s["scale"]
                x[hidden] = -math.inf
                lse[a:a + m, i] = torch.logsumexp(x, 1)
                o[a:a + m, i] = torch.softmax(x, 1) @ v
    return o, lse
