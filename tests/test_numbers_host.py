"""Whole numbers that the C entry points take as 32 bits: one that does not fit
is refused by name of its value, before anything else is looked at, and none of
its bits are dropped (no kernel launched; the tensors are on the host, which the
calls refuse next)."""
import pytest
import torch

mod = pytest.importorskip("expert_grouping_dispatch_amd")

X, Q, S = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
F8, F8S = torch.zeros(2, 32).to(torch.float8_e4m3fn), torch.zeros(2, 1)
I, U = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32).view(torch.uint32)
CALLS = {
    "mask": lambda tp_rank=0: mod.moe_mask_padding(I, I, tp_rank),
    "indices": lambda n_experts=1, scales_align=8: mod.moe_create_indices(I, n_experts, U, U, U, I, U, Q, None, scales_align),
    "noalloc": lambda n_experts=1, scales_align=8: mod.moe_create_indices_noalloc(I, n_experts, U, U, U, I, U, None, scales_align),
    "mask_indices": lambda tp_rank=0, n_experts=1, scales_align=8: mod.moe_mask_create_indices(
        I, I, tp_rank, n_experts, U, U, U, I, U, Q, None, scales_align),
    "dispatch": lambda top_k=1: mod.moe_dispatch(X, top_k, U, X),
    "mxfp4": lambda top_k=1, flags=0: mod.moe_dispatch_mxfp4(X, top_k, U, Q, Q, flags),
    "combine": lambda top_k=1: mod.moe_combine(X, S, U, top_k, X),
    "epilogue": lambda top_k=1: mod.moe_combine_epilogue(X, S, U, top_k, X),
    "dispatch_i8": lambda top_k=1: mod.moe_dispatch_i8(X, top_k, U, Q, S),
    "matmul_i8": lambda flags=0: mod.moe_expert_matmul_i8(Q, S, U, I, Q, S, X, flags=flags),
    "layer": lambda tp_rank=0: mod.moe_layer_few(X, I, F8S, X, X, X, Q, tp_rank=tp_rank),
    "layer_f8": lambda tp_rank=0: mod.moe_layer_few(X, I, F8S, F8, F8, X, Q, F8S, F8S, tp_rank=tp_rank),
    "dispatch_f8": lambda top_k=1: mod.moe_dispatch_f8(X, top_k, U, F8, F8S),
    "matmul": lambda flags=0: mod.moe_expert_matmul(X, U, I, X, X, flags=flags),
    "matmul_f8": lambda flags=0: mod.moe_expert_matmul_f8(F8, F8S, U, I, F8, F8S, X, flags=flags),
}
NUMBERS = [(call, name) for call, f in CALLS.items() for name in f.__code__.co_varnames]


@pytest.mark.parametrize("call, name", NUMBERS)
def test_numbers_that_do_not_fit_are_refused(call, name):
    for v in (2 ** 32, 2 ** 32 + 1, 2 ** 33 + 2, 2 ** 64, -2 ** 31 - 1, -2 ** 32 + 1):
        with pytest.raises(ValueError, match=f"^{v} does not fit 32 bits"):
            CALLS[call](**{name: v})
    for v in (1, 1.0, torch.tensor(1)):  # what int() takes goes on to the next check
        with pytest.raises(ValueError, match="HIP device"):
            CALLS[call](**{name: v})


def test_sizes_that_do_not_fit_have_no_workspace():
    for f, good in ((mod.moe_create_indices_workspace_bytes, (100, 8)), (mod.moe_layer_few_workspace_bytes, (4, 2, 48))):
        assert f(*good) > 0
        for at in range(len(good)):
            for more in (2 ** 32, 2 ** 64, -2 ** 32, -2 ** 64):
                bad = list(good)
                bad[at] += more
                assert f(*bad) == 0, bad
    for n, e in ((100, 2 ** 32 + 8), (2 ** 64 + 100, 8)):
        with pytest.raises(ValueError):
            mod.alloc_indices(n, e, "cpu")
    with pytest.raises(ValueError):
        mod.alloc_layer_few(4, 2 ** 32 + 2, 48, "cpu")
