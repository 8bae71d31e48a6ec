"""What is measured of the decode step's attention side: the rotation and norm of query and key heads, the append
to a paged key-value cache, and attention of a batch over that cache with shared prefixes read once.

Every operator has a plain form (elementary torch operations in 32 bits, angles in 64) and the library's call.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
# query heads, key-value heads, head dimension: the two decoder layers of workloads/ (32 / 8 / 128), and generic ones with
# another ratio (7, 16 and 1 query heads to a key-value head) and other head dimensions
HEADS = ((32, 8, 128), (16, 8, 128), (28, 4, 128), (64, 8, 64), (16, 1, 128), (10, 10, 64), (20, 4, 96), (8, 2, 256),
         (10, 5, 192))
PAGES = (16, 32, 64, 128)


def listed():
    """Norm and append in the sizes of a decode step, an odd batch and a long prompt; attention from the smallest step to
    the longest context and the largest batch."""
    return [
        # one generated token, one sequence: the call's latency is what counts
        dict(name="norm_rope_step", op="norm_rope", tokens=1, hq=32, hkv=8, d=128, dims=128, style="half", start=511,
             norm=True),
        # an odd batch, half of each head rotated, neighbouring components as pairs, far positions
        dict(name="norm_rope_batch_37", op="norm_rope", tokens=37, hq=20, hkv=4, d=96, dims=48, style="pairs",
             start=1000003, norm=True),
        # a long prompt's queries and keys
        dict(name="norm_rope_prompt_16384", op="norm_rope", tokens=16384, hq=32, hkv=8, d=128, dims=128, style="half",
             start=0, norm=True),
        # one token of one sequence into the cache, its queries turned in the same call
        dict(name="append_step", op="append", seqs=1, new=1, context=512, pad=0, hq=32, hkv=8, d=128, dims=128,
             style="half", page=64, norm=True),
        # a batch of 48 rows, five of them padding, keys without norm, no queries in the call
        dict(name="append_batch_48", op="append", seqs=48, new=1, context=4001, pad=5, hq=0, hkv=8, d=64, dims=64,
             style="pairs", page=32, norm=False),
        # five ragged prompts at once
        dict(name="append_prompts", op="append", seqs=5, new=5000, context=77, pad=0, hq=32, hkv=8, d=128, dims=128,
             style="half", page=64, norm=True),
        # the single-sequence decode step: 512 positions
        dict(name="attend_step_512", op="attend", rows=1, groups=0, shared=0, private=512, ragged=False, hq=32, hkv=8,
             d=128, page=64),
        # one sequence with a very long context of odd length
        dict(name="attend_long_131071", op="attend", rows=1, groups=0, shared=0, private=131071, ragged=False, hq=32,
             hkv=8, d=128, page=64),
        # eight continuations of one prompt
        dict(name="attend_beams_8", op="attend", rows=8, groups=1, shared=4096, private=130, ragged=True, hq=32, hkv=8,
             d=128, page=64),
        # a server's batch behind one long system prompt
        dict(name="attend_prompt_64", op="attend", rows=64, groups=1, shared=16384, private=1024, ragged=True, hq=32,
             hkv=8, d=128, page=64),
        # six documents, sixteen questions each, seven query heads to a key-value head, small pages
        dict(name="attend_groups_96", op="attend", rows=96, groups=6, shared=6000, private=700, ragged=True, hq=28,
             hkv=4, d=128, page=16),
        # nothing shared, ragged lengths with an empty row, small heads
        dict(name="attend_ragged_48", op="attend", rows=48, groups=0, shared=0, private=8191, ragged=True, hq=64,
             hkv=8, d=64, page=32),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "attend", "attend"))
    hq, hkv, d = rng.choice(HEADS)
    dims = rng.choice((d, d, d // 2 // 16 * 16))
    style = rng.choice(("half", "pairs"))
    if op == "norm_rope":
        most = 16384 * 40 * 128 // ((hq + hkv) * d)   # no dearer than the listed prompt
        return dict(op=op, tokens=_log(rng, 1, most), hq=hq, hkv=hkv, d=d, dims=dims, style=style,
                    start=_log(rng, 1, 1 << 20) - 1, norm=rng.random() < 0.7)
    if op == "append":
        most = 12000 * 48 * 128 // ((hq + 2 * hkv) * d)
        seqs = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, new=_log(rng, 1, max(1, most // seqs)), context=_log(rng, 1, 20000), pad=rng.choice((0, 3)),
                    hq=rng.choice((0, hq)), hkv=hkv, d=d, dims=dims, style=style, page=rng.choice(PAGES),
                    norm=rng.random() < 0.7)
    rows = _log(rng, 1, 128)
    most = 131072 * 8 * 128 // (hkv * d)              # tokens of the cache, no more than the longest listed
    groups = min(rows, rng.choice((0, 1, 1, 2, 5)))
    private = _log(rng, 1, max(1, min(8192, most // 2 // rows)))
    # no more products than the listed server's batch has
    products = 64 * 16384 * 32 * 128
    shared = _log(rng, 64, max(64, min(16384, most // 2 // max(1, groups), products // (rows * hq * d)))) if groups else 0
    return dict(op=op, rows=rows, groups=groups, shared=shared, private=private, ragged=rng.random() < 0.7, hq=hq,
                hkv=hkv, d=d, page=rng.choice(PAGES))


def _spread(n, most, least=0):
    """n lengths from `least` to `most`, the largest and the smallest among them: a fixed ragged pattern."""
    u = (np.arange(n, dtype=np.uint64) * np.uint64(2654435761) % np.uint64(1 << 32)).astype(np.float64) / 2 ** 32
    v = (least + np.floor(u * (most - least + 1))).astype(np.int64)
    v[-1] = most
    return v


def _shape(case):
    """Lengths of a case (the same for every seed): for attention (shared length of each group, rows of each group,
    private tokens of each row), for the append (tokens of each sequence)."""
    if case["op"] == "append":
        n, new = case["seqs"], case["new"]
        return np.full(n, 1) if new == 1 else _spread(n, new, max(1, new // 4))
    B, G = case["rows"], case["groups"]
    private = _spread(B, case["private"]) if case["ragged"] else np.full(B, case["private"])
    if not G:
        return np.zeros(0, np.int64), np.zeros(1, np.int64), private
    shared = _spread(G, case["shared"], case["shared"] // 2) if case["ragged"] else np.full(G, case["shared"])
    shared = shared // case["page"] * case["page"]      # whole pages are shared
    return shared, np.arange(G + 1) * B // G, private


def work(case):
    d, hkv, hq = case["d"], case["hkv"], case["hq"]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (hq + hkv) * d
        return {"bytes": 4.0 * n + 4 * case["tokens"], "flops": (4.0 if case["norm"] else 0) * n + 3.0 * n * case["dims"] / d}
    if case["op"] == "append":
        t = float(_shape(case).sum() - min(case["pad"], case["seqs"] - 1) * (case["new"] == 1))
        n = t * (hq + hkv) * d
        return {"bytes": 4.0 * t * (hq + 2 * hkv) * d + 8 * t,
                "flops": (4.0 if case["norm"] else 0) * n + 3.0 * n * case["dims"] / d}
    shared, start, private = _shape(case)
    seen = private.astype(np.float64)
    for g in range(len(shared)):
        seen[start[g]:start[g + 1]] += shared[g]
    tokens = float(shared.sum() + private.sum())
    return {"bytes": 4.0 * tokens * hkv * d + 4.0 * case["rows"] * hq * d, "flops": 4.0 * float(seen.sum()) * hq * d}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _head_inputs(case, g):
    d = case["d"]
    freqs = (10000.0 ** (-torch.arange(0, case["dims"], 2, dtype=torch.float64) / case["dims"])).float().cuda()
    s = {"freqs": freqs}
    for n in "qk":
        s[n + "_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = np.random.default_rng(seed)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    s = {"case": case}
    if case["op"] == "norm_rope":
        t = case["tokens"]
        # queries, keys and values as one projection's output, the rows of a token side by side
        qkv = _normal(g, t, (hq + 2 * hkv) * d)
        s.update(_head_inputs(case, g), q=qkv[:, :hq * d].view(t, hq, d), k=qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
                 positions=_dev(case["start"] + np.arange(t)))
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
    elif case["op"] == "append":
        new = _shape(case)
        n, page = case["seqs"], case["page"]
        context = _spread(n, case["context"], case["context"] // 2)
        rows = np.repeat(np.arange(n), new)
        positions = np.concatenate([c + np.arange(m) for c, m in zip(context, new)])
        if case["new"] == 1 and n > 1:                   # rows without a sequence, at the batch's end
            positions[n - min(case["pad"], n - 1):] = -1
        need = -(-(context + new) // page)               # pages of each sequence
        # the pages that the new tokens reach, spread over the cache; earlier ones hold nothing of interest here
        first = context // page
        used = int((need - first).sum())
        order = rnd.permutation(used) + 1                # page 0 is nobody's
        table = np.zeros((n, int(need.max())), np.int64) - 1
        at = 0
        for r in range(n):
            table[r, first[r]:need[r]] = order[at:at + need[r] - first[r]]
            at += need[r] - first[r]
        t = len(rows)
        qkv = _normal(g, t, (hq + 2 * hkv) * d)
        s.update(_head_inputs(case, g), q=qkv[:, :hq * d].view(t, hq, d) if hq else None,
                 k=qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d), v=qkv[:, (hq + hkv) * d:].view(t, hkv, d),
                 positions=_dev(positions), rows=_dev(rows), table=_dev(table),
                 k_pages=_normal(g, used + 1, hkv, page, d), v_pages=_normal(g, used + 1, hkv, page, d))
        s["q_out"] = torch.zeros_like(s["q"]) if hq else None
    else:
        shared, start, private = _shape(case)
        B, page = case["rows"], case["page"]
        of = np.full(B, -1)
        for i in range(len(shared)):
            of[start[i]:start[i + 1]] = i
        base = np.where(of >= 0, shared[np.maximum(of, 0)] if len(shared) else 0, 0)
        lengths = base + private
        need = -(-lengths // page)
        common = base // page
        used = int((shared // page).sum() + (need - common).sum())
        order = rnd.permutation(max(1, used))
        table = np.full((B, max(1, int(need.max()))), -1, np.int64)
        at = 0
        for i in range(len(shared)):
            n = shared[i] // page
            table[start[i]:start[i + 1], :n] = order[at:at + n]
            at += n
        for r in range(B):
            n = need[r] - common[r]
            table[r, common[r]:need[r]] = order[at:at + n]
            at += n
        s.update(q=_normal(g, B, hq, d), out=torch.zeros((B, hq, d), dtype=torch.bfloat16, device="cuda"),
                 table=_dev(table), lengths=_dev(lengths), scale=1 / math.sqrt(d),
                 group_start=_dev(start) if len(shared) else None, shared=_dev(shared) if len(shared) else None,
                 k_pages=_normal(g, max(1, used), hkv, page, d), v_pages=_normal(g, max(1, used), hkv, page, d))
    if own:
        s["call"] = _marshal(s)
    return s


def _marshal(s):
    """The library's call with its arguments, as a program keeps it from step to step."""
    import decode_gemv_byte_amd as nwc
    case = s["case"]
    if case["op"] == "norm_rope":
        return nwc.QkNormRope(s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"], q_weight=s["q_weight"],
                              k_weight=s["k_weight"], eps=EPS, freqs=s["freqs"], style=case["style"])
    cache = nwc.PagedCache(s["k_pages"], s["v_pages"])
    if case["op"] == "append":
        return nwc.KvAppend(cache, s["table"], s["k"], s["v"], s["positions"], rows=s["rows"], k_weight=s["k_weight"],
                            q=s["q"], q_out=s["q_out"], q_weight=s["q_weight"] if case["hq"] else None, eps=EPS,
                            freqs=s["freqs"], style=case["style"])
    ws = torch.zeros(nwc.nwc_attend_workspace_size(cache, case["rows"], case["hq"], case["groups"]), dtype=torch.uint8,
                     device="cuda")
    return nwc.Attend(cache, s["table"], s["lengths"], s["q"], s["out"], ws, scale=s["scale"],
                      group_start=s["group_start"], shared_len=s["shared"])


# ------------------------------------------------------------- plain forms ---

def _turned(x, weight, positions, freqs, style):
    """Heads x [tokens, heads, d] normed and turned, in 32 bits (angles in 64)."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    angle = positions.double()[:, None, None] * freqs.double()
    c, s = angle.cos().float(), angle.sin().float()
    n = 2 * freqs.numel()
    if style == "half":
        a, b = x[..., :n // 2], x[..., n // 2:n]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((turned, x[..., n:]), -1).to(torch.bfloat16)


def _plain_append(s):
    case = s["case"]
    page = case["page"]
    valid = s["positions"] >= 0
    at = s["positions"].clamp(min=0).long()
    pages = torch.where(valid, s["table"][s["rows"].long(), at // page].long(), 0)
    slot = at % page
    keep = valid[:, None, None]
    for name, new in (("k_pages", _turned(s["k"], s["k_weight"], at, s["freqs"], case["style"])), ("v_pages", s["v"])):
        # a token without a position puts back what page 0 holds
        s[name][pages, :, slot] = torch.where(keep, new, s[name][pages, :, slot])
    if s["q"] is not None:
        s["q_out"].copy_(torch.where(keep, _turned(s["q"], s["q_weight"], at, s["freqs"], case["style"]), s["q_out"]))


def _plain_attend(s):
    case = s["case"]
    B, hkv, d = case["rows"], case["hkv"], case["d"]
    pages = s["table"].clamp(min=0).long()
    k, v = (s[n][pages].transpose(1, 2).reshape(B, hkv, -1, d).float() for n in ("k_pages", "v_pages"))
    q = s["q"].float().view(B, hkv, -1, d)
    score = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    seen = torch.arange(k.shape[2], device="cuda") < s["lengths"][:, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)     # a row that sees nothing: zeros
    s["out"].copy_(out.view(B, -1, d))


def run(s):
    op = s["case"]["op"]
    if own:
        import decode_gemv_byte_amd as nwc
        {"norm_rope": nwc.nwc_qk_norm_rope, "append": nwc.nwc_kv_append, "attend": nwc.nwc_attend}[op](s["call"])
    elif op == "norm_rope":
        for n in "qk":
            s[n + "_out"].copy_(_turned(s[n], s[n + "_weight"], s["positions"], s["freqs"], s["case"]["style"]))
    elif op == "append":
        _plain_append(s)
    else:
        _plain_attend(s)
    if op == "norm_rope":
        return s["q_out"], s["k_out"]
    return (s["k_pages"], s["v_pages"], s["q_out"]) if op == "append" else s["out"]


# ----------------------------------------------------- the definition, 64 bits ---

def _exact_heads(x, weight, positions, freqs, style):
    """Each pair of components as a complex number, times exp(i position freq)."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    out = x.clone()
    m = freqs.numel()
    first, second = (slice(0, m), slice(m, 2 * m)) if style == "half" else (slice(0, 2 * m, 2), slice(1, 2 * m, 2))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous())
    phi = torch.outer(positions.double(), freqs.double())
    z = z * torch.polar(torch.ones_like(phi), phi)[:, None]
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return tuple(_exact_heads(s[n], s[n + "_weight"], s["positions"], s["freqs"], case["style"]) for n in "qk")
    if case["op"] == "append":
        ok = (s["positions"] >= 0).nonzero()[:, 0]
        pos, row = s["positions"][ok].long(), s["rows"][ok].long()
        where = s["table"][row, pos // case["page"]].long(), pos % case["page"]
        k, v = s["k_pages"].double(), s["v_pages"].double()
        k[where[0], :, where[1]] = _exact_heads(s["k"][ok], s["k_weight"], pos, s["freqs"], case["style"])
        v[where[0], :, where[1]] = s["v"][ok].double()
        if s["q"] is None:
            return k, v, None
        q = s["q_out"].double()
        q[ok] = _exact_heads(s["q"][ok], s["q_weight"], pos, s["freqs"], case["style"])
        return k, v, q
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    ratio = case["hq"] // case["hkv"]
    for r, n in enumerate(s["lengths"].tolist()):
        if n:
            at = torch.arange(n, device="cuda")
            page = s["table"][r].long()[at // case["page"]]
            # [key-value head, token, d]
            k, v = (s[name][page, :, at % case["page"]].double().transpose(0, 1).contiguous() for name in ("k_pages", "v_pages"))
            for h in range(case["hkv"]):
                q = s["q"][r, h * ratio:(h + 1) * ratio].double()
                w = torch.softmax((k[h] @ q.T) * s["scale"], 0)
                out[r, h * ratio:(h + 1) * ratio] = w.T @ v[h]
    return out
