"""The library as it is built."""
import os

from tensor_transformer_linear_column_b200 import build_lib


def test_the_kernels_are_stored_uncompressed():
    # a program's first call waits for them, half as long again for a compressed image
    build_lib.build()
    assert "--no-compress" in build_lib.CUDA_FLAGS
    assert os.path.getsize(build_lib.LIB_PATH) > 8 << 20
