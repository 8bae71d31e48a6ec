"""A prompt's tokens, behind earlier ones, through a two-layer Llama-3.1-8B-shaped
stack (hidden 4096, 32 query / 8 key-value heads of 128, MLP 14336) to their scores:
embedding rows (nwc_gather_rows), per layer the residual sum with the norm behind it
(nwc_residual_norm), q/k/v, rotation and append to the paged cache (nwc_kv_append),
attention of the chunk (nwc_attend_chunk), o, residual sum and norm, gate/up, SiLU *
up, down; then the last norm, the LM head and nwc_token_logprobs.  The projections run
compressed (nwc_gemm_prefill).  Beside it the same step with the norms, sums, rotation,
append, attention and scores as torch operations."""
import math

import pytest
import torch

import decode_gemv_byte_amd as nwc
import workloads

L, H, HQ, HKV, D, PAGE, EPS, TOP, VOCAB, MLP = 2, 4096, 32, 8, 128, 64, 1e-5, 5, 8192, 14336
NAMES = ["q", "k", "v", "o", "gate", "up", "down"]


@pytest.fixture(scope="module")
def blobs():
    blob = {n: nwc.nwc_encode(workloads.weights(3, n)) for n in NAMES}
    blob["head"] = nwc.nwc_encode(workloads.weights(5, "lm_head", rows=slice(0, VOCAB)))
    return {n: (nwc.nwc_inspect(b), torch.from_numpy(b).cuda()) for n, b in blob.items()}


class Step:
    """One prompt's buffers and the step over them, by the library's kernels or by torch."""

    def __init__(self, blobs, tokens, context):
        self.blobs, self.T, self.length = blobs, tokens, context + tokens
        g = torch.Generator(device="cuda").manual_seed(5)
        bf, dev, T = torch.bfloat16, "cuda", tokens
        n_pages = -(-self.length // PAGE)
        self.pool = torch.randn((n_pages, L, 2, HKV, PAGE, D), generator=g, device=dev).to(bf)
        self.table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).view(1, -1).to(dev)
        self.positions = torch.arange(context, self.length, dtype=torch.int32, device=dev)
        self.rows = torch.zeros(T, dtype=torch.int32, device=dev)
        self.start = torch.tensor([0, T], dtype=torch.int32, device=dev)
        self.lengths = torch.tensor([self.length], dtype=torch.int32, device=dev)
        self.freqs = (5e5 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(dev)
        self.weights = [(1 + 0.1 * torch.randn(H, generator=g, device=dev)).to(bf) for _ in range(2 * L + 1)]
        ids = torch.randint(0, VOCAB, (T + 1,), generator=g, device=dev, dtype=torch.int32)
        self.ids, self.targets = ids[:T], ids[1:].view(T, 1).clone()
        self.buf = {n: torch.empty((T, blobs[n][0].rows), dtype=bf, device=dev) for n in NAMES}
        self.x, self.h = (torch.empty((T, H), dtype=bf, device=dev) for _ in range(2))
        self.act = torch.empty((T, MLP), dtype=bf, device=dev)
        self.att = torch.empty((T, HQ, D), dtype=bf, device=dev)
        self.logits = torch.empty((T, VOCAB), dtype=bf, device=dev)
        self.q, self.k, self.v = (self.buf[n].view(T, -1, D) for n in "qkv")
        caches = [nwc.PagedCache(self.pool[:, l, 0], self.pool[:, l, 1]) for l in range(L)]
        self.ws = torch.empty(max(nwc.nwc_prefill_workspace_size(i) for i, _ in blobs.values()), dtype=torch.uint8, device=dev)
        ws_att = torch.empty(nwc.nwc_attend_chunk_workspace_size(caches[0], 1, T, HQ), dtype=torch.uint8, device=dev)
        ws_lp = torch.empty(nwc.nwc_token_logprobs_workspace_size(T, VOCAB, TOP), dtype=torch.uint8, device=dev)
        self.blas = nwc.Blas()
        self.score = {"logprobs": torch.empty((T, 1), device=dev), "entropy": torch.empty(T, device=dev),
                      "top_ids": torch.empty((T, TOP), dtype=torch.int32, device=dev),
                      "top_logprobs": torch.empty((T, TOP), device=dev)}
        self.appends = [nwc.KvAppend(c, self.table, self.k, self.v, self.positions, rows=self.rows, q=self.q, eps=EPS,
                                     freqs=self.freqs) for c in caches]
        self.attends = [nwc.AttendChunk(c, self.table, self.start, self.lengths, self.q, self.att, ws_att) for c in caches]
        # the norm before a block, with the sum of the block before it: none before the first
        self.norms = [nwc.ResidualNorm(self.x, None if i == 0 else self.buf["down" if i % 2 == 0 else "o"], out=self.h,
                                       weight=self.weights[i], eps=EPS) for i in range(2 * L + 1)]
        self.scoring = nwc.TokenLogprobs(self.logits, ws_lp, targets=self.targets, **self.score)

    def project(self, x, *names):
        for n in names:
            nwc.nwc_gemm_prefill(self.blas, *self.blobs[n], x, self.logits if n == "head" else self.buf[n], self.ws)

    def turned(self, t):
        angle = self.positions.double()[:, None, None] * self.freqs.double()
        cos, sin = angle.cos().float(), angle.sin().float()
        a, b = t.float().split(D // 2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(torch.bfloat16)

    def torch_attention(self, l):
        slots, pages = (self.positions % PAGE).long(), self.table[0, (self.positions // PAGE).long()].long()
        late = torch.arange(self.length, device="cuda")[None] > self.positions[:, None]
        self.pool[pages, l, 0, :, slots] = self.turned(self.k)
        self.pool[pages, l, 1, :, slots] = self.v
        k, v = (self.pool[:, l, i][self.table[0].long()].transpose(0, 1).reshape(HKV, -1, D)[:, :self.length].float() for i in (0, 1))
        q = self.turned(self.q).float().view(self.T, HKV, -1, D)
        for j in range(HKV):
            s = torch.matmul(q[:, j].transpose(0, 1), k[j].T.contiguous()) * D ** -0.5
            w = torch.softmax(s.masked_fill(late, -math.inf), -1)
            self.att[:, j * 4:(j + 1) * 4] = torch.matmul(w, v[j]).transpose(0, 1)

    def norm(self, i, ours):
        if ours:
            return nwc.nwc_residual_norm(self.norms[i])
        if i:
            self.x.add_(self.buf["down" if i % 2 == 0 else "o"])
        self.h.copy_(torch.nn.functional.rms_norm(self.x, (H,), self.weights[i], eps=EPS))

    def run(self, ours):
        nwc.nwc_gather_rows(*self.blobs["head"], self.ids, self.x)
        for l in range(L):
            self.norm(2 * l, ours)
            self.project(self.h, "q", "k", "v")
            if ours:
                nwc.nwc_kv_append(self.appends[l])
                nwc.nwc_attend_chunk(self.attends[l])
            else:
                self.torch_attention(l)
            self.project(self.att.view(self.T, -1), "o")
            self.norm(2 * l + 1, ours)
            self.project(self.h, "gate", "up")
            torch.mul(torch.nn.functional.silu(self.buf["gate"]), self.buf["up"], out=self.act)
            self.project(self.act, "down")
        self.norm(2 * L, ours)
        self.project(self.h, "head")
        if ours:
            nwc.nwc_token_logprobs(self.scoring)
        torch.cuda.synchronize()
        return {"hidden": self.h.double(), "logits": self.logits.double(), **{n: t.clone() for n, t in self.score.items()}}


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,context", [(70, 130), (200, 0), (33, 1001)])
def test_prompt_step_tracks_torch(blobs, tokens, context):
    step = Step(blobs, tokens, context)
    a, again, b = step.run(True), step.run(True), step.run(False)
    assert all(torch.equal(a[n], again[n]) for n in a)
    # every BF16 tensor on the way may come out a rounding apart on either side (per layer: norm, queries and keys turned,
    # attention with its weights' rounding, o, x, norm, gate and up with the activation, down, x; and the last norm: 2 * 10 + 1).
    # A rounding error is uniform within half a step, 2^-8 of the value at most, so its mean square is at most 2^-16 / 3; two
    # stacks of 21 roundings with errors of their own are sqrt(2 * 21 / 3) 2^-8 apart in the norm
    assert float((a["hidden"] - b["hidden"]).norm() / b["hidden"].norm()) < (2 * 21 / 3) ** 0.5 * 2 ** -8
    # 8192 logits of ordinary size: see the bound of the log probabilities' own test, 2^-24 (2 + 64) + 2^-21 (64 + 10 + 1)
    exact = torch.log_softmax(a["logits"], -1)
    tol = 2 ** -24 * 66 + 2 ** -21 * 75
    assert float((a["logprobs"] - exact.gather(1, step.targets.long())).abs().max()) < tol
    assert float((a["entropy"] + (exact.exp() * exact).sum(-1)).abs().max()) < 16 * tol  # weights of log weights, 10 at most, sum to 1
    assert float((a["top_logprobs"] - exact.topk(TOP, -1).values).abs().max()) < tol
    # of equal logits the one of the lower index first
    order = torch.sort(a["logits"], dim=-1, descending=True, stable=True).indices[:, :TOP]
    assert torch.equal(a["top_ids"].long(), order)
