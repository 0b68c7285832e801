"""The recurrence of linear attention in 64 bits on the device, token by token, for the GPU tests of sizes
that are slow in numpy."""
import torch


def recurrence(c, S0=True, q_scale=0.5, absolute=False):
    """(o [T, H, dv], S [B, H, dv, dk]) of a case of test_gpu_linear_attn.make, as float64 numpy arrays;
    rows of no prompt are zero.  ``absolute``: of the inputs' absolute values."""
    q, k, v, alpha = (c[n].double().abs() if absolute else c[n].double() for n in ("q", "k", "v", "alpha"))
    T, H, dv = v.shape
    group = H // q.shape[1]
    q, k = q.repeat_interleave(group, 1) * q_scale, k.repeat_interleave(group, 1)
    alpha = alpha.expand(T, H)
    S = c["S0"].double().clone() if S0 else torch.zeros(c["S0"].shape, dtype=torch.float64, device=v.device)
    if absolute:
        S.abs_()
    o = torch.zeros(T, H, dv, dtype=torch.float64, device=v.device)
    cu = c["cu"].tolist()
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            S[b] = alpha[t][:, None, None] * S[b] + v[t][:, :, None] * k[t][:, None, :]
            o[t] = (S[b] @ q[t][:, :, None])[:, :, 0]
    return o.cpu().numpy(), S.cpu().numpy()
