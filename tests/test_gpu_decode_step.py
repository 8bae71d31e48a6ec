"""A whole decode step through a two-layer Qwen3-4B-shaped stack, captured in
a HIP graph: the stack with compressed projections must track the same stack
on the dense BF16 weights (the products differ only in rounding order), and
every graph replay must reproduce the eager step's bits."""
import argparse

import pytest


@pytest.mark.gpu
def test_decode_step_stack_tracks_dense_and_replays_exactly():
    import bench
    r = bench.model_step(argparse.Namespace(model_step=2, steps=3, warmup=1))
    assert r["config"]["layers"] == 2
    # per element the two stacks may round a projection output one BF16 ulp
    # (2^-8 relative) apart; over the hidden vector the norm-relative gap
    # stays far below that after two layers
    assert r["final_hidden_rel_diff_vs_dense"] < 2 ** -8
    assert r["graph_replays_match_eager"] == {"compressed": True, "dense": True}
    assert r["value"] > 0 and r["dense_bf16_torch_mv"]["tokens_per_s"] > 0
    assert r["weight_bytes"]["compressed"] < 0.8 * r["weight_bytes"]["bf16"]


@pytest.mark.gpu
@pytest.mark.parametrize("batch,context,prefix", [(1, 130, 0), (6, 70, 1024)])
def test_paged_decode_step_tracks_torch_and_replays_exactly(batch, context, prefix):
    import bench
    r = bench.model_step_paged(argparse.Namespace(model_step=2, steps=3, warmup=1, batch=batch, context=context, prefix=prefix))
    # the steps compute the same numbers up to FP32 rounding and the rounding of the attention weights, so every BF16 tensor
    # on the way (per layer: attention, o, x, norm, gate, up with the activation, down, x: 16 in two layers) may come out a
    # rounding apart.  A rounding error is uniform within half a step, 2^-8 of the value at most, so its mean square is at
    # most 2^-16 / 3; two stacks of 16 roundings with errors of their own are sqrt(2 * 16 / 3) 2^-8 apart in the norm
    assert r["final_hidden_rel_diff"] < (2 * 16 / 3) ** 0.5 * 2 ** -8
    assert r["graph_replays_match_eager"]["ours"]
    assert r["value"] > 0 and r["config"]["batch"] == batch
