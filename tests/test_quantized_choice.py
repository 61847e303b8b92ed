"""Every variant of the int8 product's kernels and of the rows' kernels has a size among those that the GPU tests run."""
import kernel_choice as kc
import quantized_sizes as sizes


def test_every_kernel_of_the_int8_product_has_a_size():
    got = {kc.int8_product(M, N, K, g, N % 4 == 0, rows16)[0] for M, N, K, g, rows16 in sizes.products()}
    assert kc.int8_product_kernels() - got == set()


def test_every_kernel_of_the_rows_has_a_size():
    got = {kc.rows_kernel(rows, H, x, r, y, codes) for rows, H, x, r, y, codes in sizes.norms()}
    got |= {kc.rows_kernel(rows, K, x, norm=False) for rows, K, x in sizes.quantisers()}
    assert kc.rows_kernels() - got == set()


def test_the_choice_of_some_products():
    """As the launcher's traces have it."""
    assert kc.int8_product(6000, 4096, 4096)[0] == ("tile", 4, "whole", True, False)
    assert kc.int8_product(1, 1536, 4096, gated=True)[0] == ("stream", (1, 1), True)
    assert kc.int8_product(16, 4096, 1536)[0] == ("rows", (1, 2), "whole", True, False)
    assert kc.int8_product(128, 4096, 4096)[0] == ("rows", (2, 4), "whole", True, False)
    assert kc.int8_product(1000, 1003, 1100, vec=False)[0] == ("rows", (2, 4), "part", False, False)
    assert kc.rows_kernel(6000, 4096, "bf16", "bf16", "bf16") == (True, 2, 2, True, 1024, 2)
    assert kc.rows_kernel(64, 256, "f32", None, "f32", codes=False) == (True, 4, 0, False, 32, 1)
    assert kc.rows_kernel(16384, 1536, "bf16", norm=False) == (False, 2, 0, False, 1024, 1)
