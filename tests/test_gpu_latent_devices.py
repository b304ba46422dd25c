"""The calls of the two forms of latent attention refuse every tensor that is on another device than the current one. (One GPU: a tensor
that says so stands for one that is.)"""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs

pytestmark = pytest.mark.gpu


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def calls():
    T, N, H, D = 3, 5, 2, 128
    workspace = torch.empty(hs.hs_mla_expanded_workspace_size(1, D), dtype=torch.uint8, device="cuda")
    return {
        hs.hs_kv_read: dict(kv_pool=torch.zeros((64, 656), dtype=torch.uint8, device="cuda"), block_table=i32(0)[None], out_start=i32(0, N),
                            out=bf16(N, 576), err_flag=i32(0), first=i32(0)),
        hs.hs_mla_absorb: dict(q=bf16(T, H, D), w=bf16(H, 2 * D, 512), out=bf16(T, H, 512), err_flag=i32(0)),
        hs.hs_mla_project: dict(x=bf16(T, H, 512), w=bf16(H, 2 * D, 512), out=bf16(T, H, D), err_flag=i32(0)),
        hs.hs_mla_expand: dict(latent=bf16(N, 512), w=bf16(H, 2 * D, 512), kv=bf16(N, H, 2 * D), err_flag=i32(0)),
        hs.hs_mla_expanded_fwd: dict(q=bf16(T, H, D + 64), kv=bf16(N, H, 2 * D), rope=bf16(N, 64), req_start=i32(0, T), kv_start=i32(0, N),
                                     softmax_scale=0.1, out=bf16(T, H, D), err_flag=i32(0), workspace=workspace,
                                     lse=torch.zeros((T, H), device="cuda")),
    }


@pytest.mark.parametrize("call", [hs.hs_kv_read, hs.hs_mla_absorb, hs.hs_mla_project, hs.hs_mla_expand, hs.hs_mla_expanded_fwd], ids=lambda f: f.__name__)
def test_tensors_elsewhere_are_refused(call):
    args = calls()[call]
    call(**args)
    assert hs.hs_check_flag(args["err_flag"]) == 0
    for name, t in args.items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(hs.HSError, match="another device"):
                call(**{**args, name: t.as_subclass(Elsewhere)})
