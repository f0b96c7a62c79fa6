"""Sizes that reach every kernel of the block-scaled product, and which one
each reaches on a card of 256 compute units: (outputs, tokens, parts of K) of
a workgroup, 0 parts for the kernel without LDS tiles.  tests/test_product_choice.py
asks the library's own rule, so a rule that changes cannot leave a kernel
without its tests."""

CUS = 256

# {(outputs, tokens, parts): [(M, N, K), ...]} with bf16 outputs
BF16 = {
    (16, 16, 0): [(40, 300, 272), (20, 200, 4112)],      # one block a wave at a time, and two
    (32, 16, 0): [(275, 228, 800)],
    (32, 32, 0): [(300, 520, 1024)],
    (64, 32, 0): [(518, 486, 16)],
    (64, 64, 4): [(393, 628, 4096)],
    (64, 64, 2): [(419, 591, 1024)],
    (64, 64, 1): [(1100, 1000, 512)],
    (128, 128, 2): [(700, 3000, 2560)],
    (128, 128, 1): [(4500, 4400, 272)],
    (256, 256, 1): [(5337, 5563, 432), (5400, 5600, 2192)],   # the second: three chunks of scales, a short last block
}

# ... and with fp32 outputs
FP32 = {
    (16, 16, 0): [(40, 300, 272), (20, 200, 4112)],
    (32, 16, 0): [(275, 228, 800)],
    (32, 32, 0): [(300, 520, 1024)],
    (64, 32, 0): [(518, 486, 16)],
    (64, 64, 4): [(1059, 589, 7680)],
    (64, 64, 2): [(300, 4100, 2048), (346, 11063, 1024)],     # the second: three tiles a workgroup
    (64, 64, 1): [(1000, 1002, 1008)],
    (128, 128, 2): [(700, 3000, 2560)],
    (128, 128, 1): [(5337, 5563, 432)],
}
