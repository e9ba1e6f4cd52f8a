"""A call that fails leaves nothing behind for the next one."""
import pytest
import torch

from test_serving_host import SCORE

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
from epilogue_scaled_gemm_amd import serving  # noqa: E402

pytestmark = pytest.mark.gpu

OOM = -4


def test_the_call_after_a_failed_allocation():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = lg.Handle()
    x = torch.randn(2, 60001, device="cuda")
    tok = torch.tensor([5, 60000], dtype=torch.int32, device="cuda")
    lp = torch.empty(2, device="cuda")
    want = torch.log_softmax(x.double(), -1).gather(1, tok.long()[:, None])[:, 0]
    # 2^23 rows of 2^30 logits need 9 TB of partials: refused by the allocation,
    # before anything is launched on these addresses
    d = dict(rows=1 << 23, vocab=1 << 30, row_stride=1 << 30, logits=x.data_ptr(), tokens=tok.data_ptr(),
             temperature=1.0, logprobs=lp.data_ptr(), top=32, top_ids=lp.data_ptr())
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    A, B = torch.randn(4, 512, device="cuda").bfloat16(), torch.randn(64, 512, device="cuda").bfloat16()
    calls = [lambda: h.token_logprobs(x, tok, lp), lambda: h.qk_norm_rope(q, q, q.clone(), q.clone()),
             lambda: h.run(A, B, torch.empty(4, 64, dtype=torch.bfloat16, device="cuda"))]
    for after in calls:
        rc = lg.library().lin_gemm_token_logprobs(h._h, serving._SCORE.pack(*[d.get(n, 0) for n in SCORE]),
                                                  torch.cuda.current_stream().cuda_stream)
        assert rc == OOM
        after()                             # raised LinGemmError for the error before
    lp.fill_(77)
    h.token_logprobs(x, tok, lp)
    torch.cuda.synchronize()
    assert (lp.double() - want).abs().max() < 1e-4
    h.close()
