"""One call of each training loss with its gradient, for a profiler to record."""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from vocab_log_softmax_gb300 import binding as B  # noqa: E402

CASES = [  # loss, rows, columns, dtype, softcap, targets a row
    ("policy", 1024, 151936, torch.bfloat16, 0.0, 1),
    ("policy", 4096, 30011, torch.float16, 0.0, 1),
    ("policy", 1024, 262144, torch.bfloat16, 30.0, 1),
    ("policy", 512, 151936, torch.float32, 0.0, 1),
    ("distill", 1024, 151936, torch.bfloat16, 0.0, 64),
    ("distill", 1021, 65537, torch.float32, 0.0, 256),
    ("preference", 1024, 151936, torch.bfloat16, 0.0, 1),
]


def main():
    for loss, n, v, dtype, cap, k in CASES:
        gen = torch.Generator(device="cuda").manual_seed(0)
        x = (3 * torch.randn((n, v), generator=gen, device="cuda")).to(dtype)
        ids = torch.randint(0, v, (n, k), generator=gen, device="cuda")
        f = torch.randn(n, generator=gen, device="cuda")
        grad = torch.empty((n, v), dtype=dtype, device="cuda")
        if loss == "policy":
            B.vls_policy_loss(x, ids, f - 8, f, f, f - 8, kl_coef=0.1, cap=cap, dlogits=grad)
        elif loss == "distill":
            B.vls_distill_loss(x, ids, torch.randn((n, k), generator=gen, device="cuda"), f, cap=cap, dlogits=grad)
        else:
            offsets = torch.tensor([0, n // 2, n], device="cuda")     # one pair, half the rows each
            B.vls_preference_loss(x, ids, offsets, f, cap=cap, dlogits=grad)
        torch.cuda.synchronize()


if __name__ == "__main__":
    main()
