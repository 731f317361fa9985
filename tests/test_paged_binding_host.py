"""What the paged cache's binding refuses before it reaches the library, without a GPU."""

import pytest

from mixed_precision_quantized_quant_gb300 import kvq as K


def test_config_numbers_that_do_not_fit_the_c_types():
    good = dict(layers=[(16, 16), (4, 2)], num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=32, num_pages=5)
    assert K.make_paged_config(**good).num_pages == 5
    for name, value in (("num_q_heads", 2 ** 32 + 8), ("num_kv_heads", 2 ** 32 + 2), ("head_dim", 2 ** 32 + 128), ("page_size", 2 ** 33 + 32),
                        ("num_pages", 2 ** 32 + 1), ("num_pages", 2 ** 31), ("num_pages", -2 ** 32 + 4),
                        ("layers", [(256 + 4, 2)]), ("layers", [(4, 2), (4, 512 + 2)]), ("layers", [(-252, 4)])):
        with pytest.raises(ValueError):
            K.make_paged_config(**dict(good, **{name: value}))
    with pytest.raises(ValueError):
        K.make_paged_config(**good, dtype=2 ** 32)
