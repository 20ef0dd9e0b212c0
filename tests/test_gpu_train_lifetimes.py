"""Weights that a training step lays out anew, let go of while another stream still
reads them; and codes and scales that can be let go of one without the other."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_streams import SLOW, rows, same

pytestmark = pytest.mark.gpu


def busy(stream):
    overwrite((1,))  # a kernel's first launch, which loads it, waits for the device
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(SLOW)


def overwrite(like):
    """Memory of the sizes of `like` on the current stream, written to."""
    junk = []
    for t in like:
        for _ in range(4):
            junk.append(torch.full((t,), 0x7b, dtype=torch.uint8, device="cuda"))
    return junk


@pytest.mark.parametrize("mode", ["mxfp8_b32", "fp8_block128"])
@pytest.mark.parametrize("total", [24, 4096])
def test_weights_of_a_grouped_product(mode, total):
    a, a_s = fg.quantize(mode, rows(1, total, 1024))
    b, b_s = (fg.quantize_weight if mode == "fp8_block128" else fg.quantize)(mode, rows(2, 8 * 512, 1024))
    offsets = ref.fixed_offsets([total // 8] * 8)
    want = fg.grouped_gemm(a, fg.preshuffle_b(mode, b, b_s), offsets, a_s)
    pb = fg.preshuffle_b(mode, b, b_s)
    sizes = pb.data.numel(), pb.sf.numel()
    other = torch.cuda.Stream()
    busy(other)
    got = fg.grouped_gemm(a, pb, offsets, a_s, stream=other)
    del pb
    junk = overwrite(sizes)
    torch.cuda.current_stream().synchronize()
    assert not other.query() and junk
    torch.cuda.synchronize()
    assert same((got,), (want,))


@pytest.mark.parametrize("mode", ["mxfp8_b32", "fp8_block128"])
def test_weights_on_their_way_into_the_images(mode):
    quantize = fg.quantize_weight if mode == "fp8_block128" else fg.quantize
    w = rows(3, 1024, 2048)
    parts = quantize(mode, w)
    want = fg.preshuffle_b(mode, *parts)
    sizes = parts[0].numel(), parts[1].numel() * parts[1].element_size(), parts[0].untyped_storage().nbytes()
    other = torch.cuda.Stream()
    del parts
    parts = quantize(mode, w)
    busy(other)
    got = fg.preshuffle_b(mode, *parts, stream=other)
    del parts
    junk = overwrite(sizes)
    torch.cuda.current_stream().synchronize()
    assert not other.query() and junk
    torch.cuda.synchronize()
    assert same((got.data, got.sf), (want.data, want.sf))


@pytest.mark.parametrize("mode", ["mxfp8_b32", "fp8_block128"])
def test_images_on_their_way_back(mode):
    b, b_s = (fg.quantize_weight if mode == "fp8_block128" else fg.quantize)(mode, rows(4, 1024, 2048))
    pb = fg.preshuffle_b(mode, b, b_s)
    want = fg.unshuffle_b(pb)
    sizes = pb.data.numel(), pb.sf.numel()
    other = torch.cuda.Stream()
    busy(other)
    got = fg.unshuffle_b(pb, stream=other)
    del pb
    junk = overwrite(sizes)
    torch.cuda.current_stream().synchronize()
    assert not other.query() and junk
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("mode", ["mxfp8", "mxfp8_b32", "mxfp4", "fp8_block128"])
def test_codes_and_scales_have_memory_of_their_own(mode):
    """One can be kept, saved or handed on without the other."""
    x = rows(5, 33, 1024)
    for codes, scales in (fg.quantize(mode, x), fg.quantize(mode, x, act="swiglu"),
                          fg.rmsnorm_quantize(mode, x, torch.ones(1024, device="cuda", dtype=torch.bfloat16))[:2]):
        for t in (codes, scales):
            assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size()
