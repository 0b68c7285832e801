"""Calls of two host threads at once, each on a stream and tensors of its own: the binding lets go of the interpreter's lock, so
that they meet inside the library.  Their kernels take different amounts of shared memory."""
import threading

import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
from _window import DEV, whole

pytestmark = pytest.mark.gpu


def rotation(Hq, Hkv, io, rounds):
    """A thread's work: the same call many times, without the binding's checks in between; its tensors, and what went wrong."""
    g = torch.Generator().manual_seed(Hq)
    q, k = (torch.randn(5, n, 256, generator=g).to(io).to(DEV) for n in (Hq, Hkv))
    out = [torch.zeros_like(q), torch.zeros_like(k)]
    prefix, err, failed = whole([0, 5, 9, 100, 7]), whole([9] * 5), []
    stream = torch.cuda.Stream()
    here = [t.data_ptr() for t in (q, k, *out, prefix, err)]
    args = (here[0], Hq * 256, here[1], Hkv * 256, None, Hkv * 256, None, None, None, here[4], None, 5, 5, Hq, Hkv, 256, 256,
            tv.TV_BF16 if io == torch.bfloat16 else tv.TV_F32, 1, 1e-6, 0.0, 1e4, here[2], Hq * 256, here[3], Hkv * 256, None,
            None, 0, None, 0, 0, here[5], stream.cuda_stream)

    def work():
        call = tv.lib.tv_qk_norm_rope
        failed.extend(s for s in (call(*args) for _ in range(rounds)) if s != tv.TV_OK)
        stream.synchronize()
    return work, out, err, failed, (q, k, prefix, stream)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_rotations_of_different_shapes(io):
    shapes = [(24, 8), (8, 4) if io == torch.float32 else (20, 8)]
    wants = []
    for shape in shapes:
        work, out, err, failed, _ = rotation(*shape, io, 1)
        torch.cuda.synchronize()
        work()
        assert not failed and not err.any()
        wants.append(out)
    works = [rotation(*shape, io, 30000) for shape in shapes]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=w[0]) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (_, out, err, failed, _), want in zip(works, wants):
        assert not failed, f"{len(failed)} of 30000 calls: {set(failed)}"
        assert not err.any() and all(torch.equal(a, b) for a, b in zip(out, want))
