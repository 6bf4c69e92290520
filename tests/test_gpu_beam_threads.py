"""Beam selections of different sizes from host threads at once (needs a GB300)."""
import threading

import numpy as np
import pytest
import torch

from rank_compressed_paged_gb300 import _lib, beam_select, beam_workspace_bytes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,code", [(torch.float32, _lib.RCP_LOGITS_FP32),
                                        (torch.float16, _lib.RCP_LOGITS_FP16)])
def test_selections_of_different_sizes_from_threads(dtype, code):
    """Each thread has its stream, its buffers and its size, whose merge takes 50 to 220 KB of shared
    memory, and makes the library's call over and over: none is refused, and each gives what it
    gives alone."""
    lib = _lib.load()
    sizes = [(1, 32, 2 ** 18), (1, 16, 2 ** 18), (1, 8, 2 ** 18), (1, 24, 100001)]
    cases, refused, wrong = [], [], []
    for B, K, V in sizes:
        r = np.random.default_rng(K)
        x = torch.from_numpy(3 * r.standard_normal((B, K, V))).to(dtype).cuda()
        s = torch.from_numpy(r.standard_normal((B, K)).astype(np.float32)).cuda()
        out = [torch.empty_like(s), torch.empty_like(s, dtype=torch.int32),
               torch.empty_like(s, dtype=torch.int32), torch.empty_like(s)]
        ws = torch.empty(beam_workspace_bytes(B, K, V, dtype), dtype=torch.uint8, device="cuda")
        cases.append((x, s, B, K, V, out, ws, torch.cuda.Stream(), beam_select(x, s, eos=1)))
    torch.cuda.synchronize()
    start = threading.Barrier(len(cases))

    def go(x, s, B, K, V, out, ws, stream, want):
        args = (x.data_ptr(), code, s.data_ptr(), B, K, V, 1, *(o.data_ptr() for o in out),
                ws.data_ptr(), ws.numel(), stream.cuda_stream)
        start.wait()
        for _ in range(4000):
            status = lib.rcp_beam_select(*args)
            if status != _lib.RCP_OK:
                refused.append((K, status))
                break
        stream.synchronize()
        wrong.extend(K for a, b in zip(out, want) if not torch.equal(a, b))
    threads = [threading.Thread(target=go, args=c) for c in cases]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not refused and not wrong, (refused, wrong)
