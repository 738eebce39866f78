"""The paged cache in the bounds-checked build: its device-side checks run in
every build, and this one reports a failed one as HGA_ERR_DEVICE_CHECK."""
import pytest
import torch

import hierarchical_routed_sparse_b200 as hga

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _checked_library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from hierarchical_routed_sparse_b200 import build
    build.build()
    build.build(checked=True)
    hga.use_library(hga.CHECKED_LIB_PATH)
    assert hga.checked_build()
    yield
    hga.use_library(build.LIB)
    assert not hga.checked_build()


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("k_c,k_g", [(1, 4), (-1, -1)])
def test_a_bad_page_is_reported(k_c, k_g):
    p = hga.PagedParams(1, 4, 2, 64, 4, 3, k_c, k_g)
    c = hga.PagedCache(p, table=_int32([[0, 1, 2]]))
    x = torch.randn(150, 2, 64, device="cuda").bfloat16()
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    O, lse = torch.empty(1, 4, 64, device="cuda"), torch.empty(1, 4, device="cuda")
    rows = (None, None) if k_c < 0 else (torch.empty(1, 2, k_c, dtype=torch.int32, device="cuda"),
                                         torch.empty(1, 2, k_g, dtype=torch.int32, device="cuda"))
    c.append(_int32([0]), x, x, cu=_int32([0, 150]))
    c.decode(_int32([149]), q, O, lse, *rows)
    assert torch.isfinite(O).all()
    c.table[0, 1] = 4
    for call in (lambda: c.decode(_int32([149]), q, O, lse, *rows),
                 lambda: c.append(_int32([0]), x, x, cu=_int32([0, 150])),
                 lambda: c.append(_int32([100]), x, x, cu=_int32([0, 150]))):
        with pytest.raises(hga.HGAError) as e:
            call()
        assert e.value.code == hga.HGA_ERR_DEVICE_CHECK
    c.table[0, 1] = 1
    c.decode(_int32([149]), q, O, lse, *rows)
    assert torch.isfinite(O).all() and hga.device_check() == 0


def test_a_step_past_the_end_is_reported_and_not_counted():
    st = hga.PagedDecodeState(2, 4, 2, 64, 64, 1, 4, rope=hga.rope_table(64, 64))
    x = torch.randn(2, 8, 64, device="cuda").bfloat16()
    st.pos.copy_(_int32([63, 5]))
    st.step(x[:, :4], x[:, 4:6], x[:, 6:])
    assert st.pos.tolist() == [64, 6]
    with pytest.raises(hga.HGAError) as e:
        st.step(x[:, :4], x[:, 4:6], x[:, 6:])
    assert e.value.code == hga.HGA_ERR_DEVICE_CHECK and st.pos.tolist() == [64, 6]
    with pytest.raises(hga.HGAError) as e:
        st.cache.advance(st.pos)
    assert e.value.code == hga.HGA_ERR_DEVICE_CHECK
    assert st.pos.tolist() == [64, 7] and hga.device_check() == 0
