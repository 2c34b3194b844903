// Host program under UndefinedBehaviorSanitizer: where a lane's vector of a row
// is read and how far it is shifted (span_of, settle in train_common.hpp), for
// rows of 1 to 199 values and lanes far past the row's end too.  Prints
// the number of vectors checked.
#include <cstdio>
#include <cstring>

#include "../../tensor_product_message_amd/csrc/train_common.hpp"

template <class T>
long check() {
    using namespace ctp;
    long checked = 0;
    for (int n = 1; n < 200; ++n)
        for (int v = 0; v < 1024; ++v, ++checked) {
            const Span s = span_of<T>(v, n);
            const int begin = v * kVec<T>, have = n - begin;        // values that the vector has
            // what a lane holds: the read vector, or zeros where the vector lies past the end
            vec_t<T> x = {};
            if (have > 0) {
                if (n < kVec<T>) {
                    if (s.shift != 0 || s.few != n) return -1;
                    for (int k = 0; k < s.few; ++k) x[k] = (T)(float)(k + 1);
                } else {
                    if (s.at < 0 || s.at + kVec<T> > n || s.few != 0) return -1;
                    for (int k = 0; k < kVec<T>; ++k) x[k] = (T)(float)(s.at + k + 1);
                }
            }
            settle<T>(x, s, have > 0);
            for (int k = 0; k < kVec<T>; ++k) {
                const float want = k < have ? (float)(T)(float)(begin + k + 1) : 0.0f;
                if ((float)x[k] != want) return -1;
            }
        }
    return checked;
}

int main() {
    const long a = check<float>(), b = check<__bf16>(), c = check<_Float16>();
    if (a < 0 || b < 0 || c < 0) {
        std::printf("wrong: %ld %ld %ld\n", a, b, c);
        return 1;
    }
    std::printf("checked %ld\n", a + b + c);
    return 0;
}
