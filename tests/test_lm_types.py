"""Tensors of another type than the call takes them for are refused before the
library is called."""
import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_lm_host import host_comm

N, VOCAB, WIDTH = 4, 8, 16
F32, BF16, F16, F64 = torch.float32, torch.bfloat16, torch.float16, torch.float64


def refused(fn, *args, **kw):
    with pytest.raises(TypeError, match="the call takes"):
        fn(*args, **kw, stream=0)


@pytest.mark.parametrize("wrong,dtype", [("hidden", F32), ("weight", F16), ("log_probs", BF16), ("entropy", F64),
                                         ("lse", F16), ("top_log_probs", BF16)])
def test_log_probs(wrong, dtype):
    t = {"hidden": torch.zeros(N, WIDTH, dtype=BF16), "weight": torch.zeros(VOCAB, WIDTH, dtype=BF16),
         "log_probs": torch.zeros(N), "entropy": torch.zeros(N), "lse": torch.zeros(N), "top_log_probs": torch.zeros(N, 2)}
    t[wrong] = t[wrong].to(dtype)
    refused(ar.ar_linear_log_probs, host_comm(), t["hidden"], t["weight"], torch.zeros(N, dtype=torch.int64), t["log_probs"],
            t["entropy"], t["lse"], N, VOCAB, WIDTH, "bf16", top=2, top_log_probs=t["top_log_probs"],
            top_ids=torch.zeros(N, 2, dtype=torch.int32))


@pytest.mark.parametrize("wrong,dtype", [("hidden", F32), ("weight", F16), ("lse", BF16), ("entropy", F16),
                                         ("grad_log_probs", BF16), ("grad_entropy", F64), ("grad_hidden", F32),
                                         ("grad_weight", F32)])
def test_log_probs_backward(wrong, dtype):
    names = ("lse", "entropy", "grad_log_probs", "grad_entropy")
    t = {"hidden": torch.zeros(N, WIDTH, dtype=BF16), "weight": torch.zeros(VOCAB, WIDTH, dtype=BF16),
         "grad_hidden": torch.zeros(N, WIDTH, dtype=BF16), "grad_weight": torch.zeros(VOCAB, WIDTH, dtype=BF16),
         **{k: torch.zeros(N) for k in names}}
    t[wrong] = t[wrong].to(dtype)
    refused(ar.ar_linear_log_probs_backward, host_comm(), t["hidden"], t["weight"], torch.zeros(N, dtype=torch.int64),
            *[t[k] for k in names], t["grad_hidden"], t["grad_weight"], N, VOCAB, WIDTH, "bf16")


def test_orthogonalize():
    x, y = [torch.zeros(8, 16, dtype=BF16) for _ in range(3)], [torch.zeros(8, 16, dtype=BF16) for _ in range(3)]
    refused(ar.ar_orthogonalize, host_comm(), x, y, 8, 16, "f32")
    refused(ar.ar_orthogonalize, host_comm(), x, y[:2] + [y[2].float()], 8, 16, "bf16")
    refused(ar.ar_orthogonalize, host_comm(), [x[0], x[1].half(), x[2]], y, 8, 16, "bf16")


@pytest.mark.parametrize("wrong,dtype", [("grads", F32), ("momentum_in", BF16), ("momentum_out", BF16), ("weights_in", F32),
                                         ("weights_out", F32)])
def test_muon_update(wrong, dtype):
    """fp32 weights want weight_dtype to say so; the momentum is always fp32."""
    t = {"grads": BF16, "momentum_in": F32, "momentum_out": F32, "weights_in": BF16, "weights_out": BF16}
    t[wrong] = dtype
    lists = {k: [torch.zeros(8, 16, dtype=d) for _ in range(2)] for k, d in t.items()}
    lists["weights_out"] = [[w, torch.zeros_like(w)] for w in lists["weights_out"]]
    refused(ar.ar_muon_update, host_comm(2), *lists.values(), 8, 16, "bf16")
