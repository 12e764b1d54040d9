"""Sizes that reach each instance of the linear prefill kernel, shared by the
GPU tests and the host test that checks the choice."""

# dk, dv, heads, key heads: heads of a key head go together 4 (dv 32), 2 (dv 64)
# or 1 to a workgroup
DIMS = [(dk, dv, H, Hk) for dk in (32, 64, 128)
        for dv, H, Hk in ((32, 4, 1), (32, 3, 3), (64, 4, 2), (64, 3, 3), (128, 2, 1))]

# "few": at most 64 tokens a sequence on average and no sequence split (chunks of
# 32 in bf16); "whole": longer, not split; "split": segments, and their join
KINDS = [("bf16", "few"), ("bf16", "whole"), ("bf16", "split"), ("f32", "whole"), ("f32", "split")]


def heads_a_workgroup(dv, H, Hk):
    most = 128 // dv
    return most if H // Hk % most == 0 else 1


def lengths_of(dtype, kind, H):
    """Below 256 sequences x heads, sequences are split from 128 tokens in all on
    (from 64 in fp32), but for bf16 batches of up to 256 tokens; from there on
    not below 1,024, and empty sequences make the number up."""
    if kind == "few":
        return [1, 31, 32, 33, 0, 64, 65, 20, 5, 2]  # 253 tokens
    if kind == "whole":
        return [190, 0, 51] if dtype == "bf16" else [300, 0, 500, 129, 65, 1] + [0] * -(-256 // H)
    return [700, 0, 1, 333]
