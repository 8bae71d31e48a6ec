"""What is measured of a step's other parts between and behind its projections: attention of a chunk of new tokens over
the paged cache, the residual stream with the norms before and after a block, and the log probabilities of given tokens
with entropy and top alternatives.

Every operator has a plain form (elementary torch operations in 32 bits) and the library's call.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
# query heads, key-value heads, head dimension: the decoder layers of workloads/ (32 / 8 / 128) and generic ones with other
# ratios (1 to 16 query heads to a key-value head) and head dimensions
HEADS = ((32, 8, 128), (32, 8, 128), (16, 8, 128), (28, 4, 128), (64, 8, 64), (16, 1, 128), (10, 10, 64), (20, 4, 96),
         (8, 2, 256), (10, 5, 192))
PAGES = (16, 32, 64, 128)
HIDDEN = (1024, 2560, 4096, 1000, 5120, 8192)      # the first three are workloads/'s
VOCABS = (128256, 128256, 32003, 50000, 1001)      # workloads/'s LM head, and generic ones, odd among them


def listed():
    """From calls whose latency counts to a document's chunk, a long prompt's residual stream and its scoring."""
    return [
        # five drafted tokens of one sequence looked over at once
        dict(name="chunk_draft_5", op="chunk", rows=1, new=5, context=507, ragged=False, singles=0, hq=32, hkv=8, d=128, page=64),
        # seven prompts of any length, some behind earlier turns, seven query heads to a key-value head, small pages
        dict(name="chunk_ragged_7", op="chunk", rows=7, new=700, context=2001, ragged=True, singles=0, hq=28, hkv=4, d=128,
             page=16),
        # a server's step: 31 sequences with one token each beside a part of one prompt, small heads
        dict(name="chunk_mixed_32", op="chunk", rows=32, new=512, context=4001, ragged=True, singles=31, hq=64, hkv=8, d=64,
             page=32),
        # a question behind a very long context
        dict(name="chunk_late_64", op="chunk", rows=1, new=64, context=131007, ragged=False, singles=0, hq=32, hkv=8, d=128,
             page=64),
        # a whole prompt
        dict(name="chunk_prompt_8192", op="chunk", rows=1, new=8192, context=0, ragged=False, singles=0, hq=32, hkv=8, d=128,
             page=64),
        # one part of a long document
        dict(name="chunk_document_4096", op="chunk", rows=1, new=4096, context=28672, ragged=False, singles=0, hq=32, hkv=8,
             d=128, page=64),
        # one generated token: the residual sum and the norm before the next block
        dict(name="norm_step", op="norm", tokens=1, cols=4096, x32=False, after=False, gate="", before=True),
        # an odd batch, the block's output normed and gated token by token, a residual stream of 32 bits
        dict(name="norm_batch_37", op="norm", tokens=37, cols=2560, x32=True, after=True, gate="tokens", before=True),
        # a long prompt
        dict(name="norm_prompt_16384", op="norm", tokens=16384, cols=4096, x32=False, after=False, gate="", before=True),
        # one generated token's log probability with its alternatives, the LM head's output in 32 bits
        dict(name="logprobs_step", op="logprobs", rows=1, vocab=128256, f32=True, targets=1, k=20, masked=False),
        # four answers compared in 16 sequences, a grammar leaving a third of an odd vocabulary
        dict(name="logprobs_answers_16", op="logprobs", rows=16, vocab=32003, f32=False, targets=4, k=5, masked=True),
        # a prompt scored token by token
        dict(name="logprobs_prompt_2048", op="logprobs", rows=2048, vocab=128256, f32=False, targets=1, k=20, masked=False),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "norm", "logprobs"))
    if op == "norm":
        cols = rng.choice(HIDDEN)
        x32, after, gate = rng.random() < 0.3, rng.random() < 0.5, rng.choice(("", "", "all", "tokens"))
        return dict(op=op, tokens=_log(rng, 1, 16384 * 4096 // (cols * (2 if x32 or after or gate else 1))), cols=cols, x32=x32,
                    after=after, gate=gate, before=rng.random() < 0.8)
    if op == "logprobs":
        vocab, f32 = rng.choice(VOCABS), rng.random() < 0.5
        rows = _log(rng, 1, min(4096, 2048 * 128256 // (vocab * (2 if f32 else 1))))
        return dict(op=op, rows=rows, vocab=vocab, f32=f32, targets=rng.choice((1, 1, 4)), k=rng.choice((0, 1, 5, 20, 50)),
                    masked=rng.random() < 0.3)
    hq, hkv, d = rng.choice(HEADS)
    rows = _log(rng, 1, 32)
    new = _log(rng, 1, 4096 // rows if rows > 1 else 8192)
    # no more products than the listed document has, no more keys and values than the listed long context
    seen = 4096 * 30720 * 32 * 128 // (rows * new * hq * d) - new // 2
    held = 131072 * 8 * 128 // (rows * hkv * d) - new * (1 + hq // hkv)
    return dict(op=op, rows=rows, new=new, context=_log(rng, 1, max(1, min(seen, held, 131072))) - 1,
                ragged=rng.random() < 0.7, singles=rng.choice((0, 0, rows // 2)), hq=hq, hkv=hkv, d=d, page=rng.choice(PAGES))


def _spread(n, most, least=0):
    """n lengths from `least` to `most`, the largest and the smallest among them: a fixed ragged pattern."""
    u = (np.arange(n, dtype=np.uint64) * np.uint64(2654435761) % np.uint64(1 << 32)).astype(np.float64) / 2 ** 32
    v = (least + np.floor(u * (most - least + 1))).astype(np.int64)
    v[-1] = most
    return v


def _shape(case):
    """New tokens and earlier positions of each row, the same for every seed; the first `singles` rows have one token."""
    n = case["rows"]
    new = _spread(n, case["new"], max(1, case["new"] // 8)) if case["ragged"] else np.full(n, case["new"])
    new[:min(case["singles"], n - 1)] = 1
    return new, _spread(n, case["context"], case["context"] // 4) if case["ragged"] else np.full(n, case["context"])


def work(case):
    if case["op"] == "norm":
        n = float(case["tokens"] * case["cols"])
        x = 4 if case["x32"] else 2
        return {"bytes": n * (2 * x + 2 + 2 * case["before"] + 2 * (case["gate"] == "tokens")),
                "flops": n * (2 + 4 * case["after"] + 4 * case["before"] + bool(case["gate"]))}
    if case["op"] == "logprobs":
        n = float(case["rows"] * case["vocab"])
        return {"bytes": n * (4 if case["f32"] else 2) + case["rows"] * (8.0 * case["targets"] + 8 * case["k"] + 4), "flops": 7 * n}
    new, context = (x.astype(np.float64) for x in _shape(case))
    pairs = float((new * context + new * (new + 1) / 2).sum())
    width = case["hq"] * case["d"]
    return {"bytes": 4.0 * float((new + context).sum()) * case["hkv"] * case["d"] + 4.0 * float(new.sum()) * width,
            "flops": 4.0 * pairs * width}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = np.random.default_rng(seed)
    s = {"case": case}
    if case["op"] == "norm":
        t, c = case["tokens"], case["cols"]
        x = 4 * torch.randn((t, c), generator=g, device="cuda")
        s["x"] = x if case["x32"] else x.to(torch.bfloat16)
        s["y"] = _normal(g, t, c)
        for name, there in (("y_weight", case["after"]), ("weight", case["before"])):
            s[name] = (1 + 0.2 * torch.randn(c, generator=g, device="cuda")).to(torch.bfloat16) if there else None
        s["gate"] = _normal(g, c) if case["gate"] == "all" else _normal(g, t, c) if case["gate"] else None
        s["scale"] = 0.22 if case["after"] else 1.0
        s["x_out"] = torch.empty_like(s["x"])
        s["out"] = torch.empty((t, c), dtype=torch.bfloat16, device="cuda") if case["before"] else None
    elif case["op"] == "logprobs":
        n, v, k = case["rows"], case["vocab"], case["k"]
        ld = -(-v // 8) * 8                              # rows of the LM head's output, 16 bytes apart
        x = torch.empty((n, ld), dtype=torch.float32 if case["f32"] else torch.bfloat16, device="cuda")
        for r in range(0, n, 256):
            part = 2.5 * torch.randn((min(256, n - r), ld), generator=g, device="cuda")
            # a few tokens far above the others, in most rows
            best = torch.randint(0, v, (len(part), 3), generator=g, device="cuda")
            part.scatter_add_(1, best, 6 + 8 * torch.rand(best.shape, generator=g, device="cuda"))
            if case["masked"]:
                part[:, torch.arange(ld, device="cuda") % 3 != 0] = -math.inf
            x[r:r + 256] = part
        s["logits"] = x[:, :v]
        step = 3 if case["masked"] else 1
        s["targets"] = _dev(rnd.integers(0, (v + step - 1) // step, (n, case["targets"])) * step)
        s["logprobs"] = torch.empty((n, case["targets"]), device="cuda")
        s["entropy"] = torch.empty(n, device="cuda")
        s["top_ids"] = torch.empty((n, k), dtype=torch.int32, device="cuda") if k else None
        s["top_logprobs"] = torch.empty((n, k), device="cuda") if k else None
    else:
        new, context = _shape(case)
        n, page, d, hq, hkv = case["rows"], case["page"], case["d"], case["hq"], case["hkv"]
        lengths = context + new
        need = -(-lengths // page)
        order = rnd.permutation(int(need.sum()))
        table = np.full((n, int(need.max())), -1, np.int64)
        at = 0
        for r in range(n):
            table[r, :need[r]] = order[at:at + need[r]]
            at += need[r]
        t = int(new.sum())
        s.update(k_pages=_normal(g, at, hkv, page, d), v_pages=_normal(g, at, hkv, page, d), q=_normal(g, t, hq, d),
                 out=torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda"), table=_dev(table), lengths=_dev(lengths),
                 query_start=_dev(np.concatenate(([0], np.cumsum(new)))), scale=1 / math.sqrt(d),
                 new=new.tolist(), context=context.tolist())
    if own:
        s["call"] = _marshal(s)
    return s


def _marshal(s):
    """The library's call with its arguments, as a program keeps it from step to step."""
    import decode_gemv_byte_amd as nwc
    case = s["case"]
    if case["op"] == "norm":
        return nwc.ResidualNorm(s["x"], s["y"], x_out=s["x_out"], out=s["out"], weight=s["weight"], y_weight=s["y_weight"],
                                gate=s["gate"], scale=s["scale"], eps=EPS)
    if case["op"] == "logprobs":
        ws = torch.zeros(nwc.nwc_token_logprobs_workspace_size(case["rows"], case["vocab"], case["k"]), dtype=torch.uint8,
                         device="cuda")
        return nwc.TokenLogprobs(s["logits"], ws, targets=s["targets"], logprobs=s["logprobs"], entropy=s["entropy"],
                                 top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    cache = nwc.PagedCache(s["k_pages"], s["v_pages"])
    ws = torch.zeros(nwc.nwc_attend_chunk_workspace_size(cache, case["rows"], s["q"].shape[0], case["hq"]), dtype=torch.uint8,
                     device="cuda")
    return nwc.AttendChunk(cache, s["table"], s["query_start"], s["lengths"], s["q"], s["out"], ws, scale=s["scale"])


# ------------------------------------------------------------- plain forms ---

def _plain_norm(s):
    def normed(v, w):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()
    u = s["y"].float()
    if s["y_weight"] is not None:
        u = normed(u, s["y_weight"])
    if s["gate"] is not None:
        u = u * s["gate"].float()
    x = s["x"].float() + s["scale"] * u
    s["x_out"].copy_(x)
    if s["out"] is not None:
        s["out"].copy_(normed(x, s["weight"]))


def _plain_logprobs(s):
    k = s["case"]["k"]
    for r in range(0, s["case"]["rows"], 512):
        x = s["logits"][r:r + 512].float()
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        total = e.sum(-1, keepdim=True)
        log_total = torch.log(total)
        s["logprobs"][r:r + 512] = x.gather(1, s["targets"][r:r + 512].long()) - m - log_total
        # a token without weight adds nothing
        s["entropy"][r:r + 512] = log_total[:, 0] + (torch.where(e > 0, e * (m - x), 0.0)).sum(-1) / total[:, 0]
        if k:
            # one whole number for value and index: the lower index is the greater of two equal values
            bits = x.view(torch.int32).long()
            key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2 ** 32 - torch.arange(x.shape[1], device="cuda")
            ids = torch.topk(key, k, -1).indices
            s["top_ids"][r:r + 512] = ids
            s["top_logprobs"][r:r + 512] = x.gather(1, ids) - m - log_total


def _plain_chunk(s):
    case = s["case"]
    hkv, hq, d = case["hkv"], case["hq"], case["d"]
    first = 0
    for r, (n, c) in enumerate(zip(s["new"], s["context"])):
        pages = s["table"][r, :-(-(c + n) // case["page"])].long()
        # [key-value head, position, d]
        k, v = (s[name][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :c + n].float() for name in ("k_pages", "v_pages"))
        step = max(1, 2 ** 29 // ((c + n) * hq))         # tokens at a time: no more than 2^29 scores
        for t in range(0, n, step):
            m = min(step, n - t)
            end = c + t + m                              # positions that the last of these tokens sees
            q = s["q"][first + t:first + t + m].float().view(m, hkv, -1, d).transpose(0, 1).reshape(hkv, -1, d)
            score = torch.matmul(q, k[:, :end].transpose(-1, -2)).view(hkv, m, -1, end) * s["scale"]
            late = torch.arange(end, device="cuda") > c + t + torch.arange(m, device="cuda")[:, None]
            score = score.masked_fill(late[:, None], -math.inf)
            e = torch.exp(score - score.amax(-1, keepdim=True))
            o = torch.matmul(e.view(hkv, -1, end), v[:, :end]).view(hkv, m, -1, d) / e.sum(-1, keepdim=True)
            s["out"][first + t:first + t + m] = o.transpose(0, 1).reshape(m, hq, d)
        first += n


def run(s):
    op = s["case"]["op"]
    if own:
        import decode_gemv_byte_amd as nwc
        {"norm": nwc.nwc_residual_norm, "logprobs": nwc.nwc_token_logprobs, "chunk": nwc.nwc_attend_chunk}[op](s["call"])
    else:
        {"norm": _plain_norm, "logprobs": _plain_logprobs, "chunk": _plain_chunk}[op](s)
    if op == "norm":
        return [s["x_out"]] + ([] if s["out"] is None else [s["out"]])
    if op == "logprobs":
        return [s["logprobs"], s["entropy"]] + ([s["top_ids"], s["top_logprobs"]] if s["case"]["k"] else [])
    return s["out"]


# ----------------------------------------------------- the definition, 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        u = s["y"].double()
        if s["y_weight"] is not None:
            u = s["y_weight"].double() * u / (u.square().sum(-1, keepdim=True) / case["cols"] + EPS).sqrt()
        if s["gate"] is not None:
            u = u * s["gate"].double()
        x = s["x"].double() + s["scale"] * u
        if s["weight"] is None:
            return [x]
        return [x, s["weight"].double() * x / (x.square().sum(-1, keepdim=True) / case["cols"] + EPS).sqrt()]
    if case["op"] == "logprobs":
        parts = []
        for r in range(0, case["rows"], 256):
            x = s["logits"][r:r + 256].double()
            lp = x - torch.logsumexp(x, -1, keepdim=True)
            p = torch.softmax(x, -1)
            part = [torch.gather(lp, 1, s["targets"][r:r + 256].long()), -(p * lp.clamp(min=-1e30)).sum(-1)]
            if case["k"]:
                top = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
                part += [top, torch.gather(lp, 1, top)]
            parts.append(part)
        return [torch.cat(p) for p in zip(*parts)]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    ratio, page = case["hq"] // case["hkv"], case["page"]
    first = 0
    for r, (n, c) in enumerate(zip(s["new"], s["context"])):
        at = torch.arange(c + n, device="cuda")
        of = s["table"][r].long()[at // page]
        for h in range(case["hkv"]):
            k, v = (s[name][of, h, at % page].double() for name in ("k_pages", "v_pages"))
            for t in range(0, n, 1024):
                pos = c + torch.arange(t, min(n, t + 1024), device="cuda")
                for j in range(h * ratio, (h + 1) * ratio):
                    score = (s["q"][first + t:first + t + len(pos), j].double() @ k.T) * s["scale"]
                    score[at[None] > pos[:, None]] = -math.inf
                    out[first + t:first + t + len(pos), j] = torch.softmax(score, -1) @ v
        first += n
    return out
