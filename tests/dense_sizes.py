"""Sizes (T, K, N) of the dense operators' tests whose bf16 products take 256 x 256 tiles for their
first output columns and a second launch for the rest; tests/test_dense_bounds.py checks that they do."""

# backward: dx and dw, of a linear and of a gated layer, with one to three terms of the gradient; the
# rest 8, 8, 904 and (in padded rows) 903 columns
CUT_BACKWARD = [(4096, 4104, 4096), (8192, 2056, 8192), (4096, 5000, 4096), (4096, 4999, 4096)]

# forward, linear
CUT_FORWARD = [(8200, 520, 4100), (8192, 200, 7168)]
