"""The workspace of a new handle is zero when create returns, whatever the memory
held and however busy the default stream is: a first call may come on a stream
that does not wait for it."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_42_gb300 import build
    build.build()
    import speculative_decoding_verification_42_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("kind", ["tree", "verify"])
def test_workspace_is_zero_for_every_stream(sv, kind):
    import torch
    blocks = []

    @sv.SPEC_ALLOC_FN
    def alloc(ctx, nbytes, device, ptr):
        t = torch.full((int(nbytes),), 255, dtype=torch.uint8, device=f"cuda:{device}")
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)  # the default stream is busy for some 100 ms
        blocks.append(t)
        ptr[0] = t.data_ptr()
        return 0

    @sv.SPEC_RELEASE_FN
    def release(ctx, ptr, device):
        pass

    side = torch.cuda.Stream()
    warm = torch.zeros(8, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        warm.any().item()  # what the read below launches is loaded
    torch.cuda.synchronize()
    sv.spec_verify_set_allocator(alloc, release)
    try:
        if kind == "tree":
            h = sv.TreeCache(max_batch=2, max_tokens=4, q_heads=4, kv_heads=2, head_dim=64, dtype="bf16",
                             page_size=16, num_pages=8, table_width=4)
        else:
            h = sv.Verifier(vocab=4096, max_batch=2, max_k=2, dtype="bf16")
    finally:
        sv.spec_verify_set_allocator(None, None)
    assert len(blocks) == 1
    with torch.cuda.stream(side):  # a stream that does not wait for the default one
        assert not blocks[0].any().item()
    torch.cuda.synchronize()
    h.close()
